"""int8 quantise and dequantise on the GPU against the definition in 64 bits: scales and codes are equal."""
import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


def pitched(x, dtype, extra=0, fill=float("nan")):
    """Device tensor of x at a pitch of 16 bytes (plus `extra` chunks); the padding holds `fill`."""
    per = 16 // SIZE[dtype]
    t = torch.full((x.shape[0], ref.up(x.shape[1], per) + extra * per), fill, dtype=DT[dtype])
    t[:, :x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    return t.cuda()


def sample(rows, cols, dtype, seed, spread=0.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * np.exp2(r.uniform(-spread, spread, (rows, cols)))
    return torch.from_numpy(x).to(DT[dtype]).double().numpy()


def quantise(g, x, dtype, k, act=qg.MX_IDENTITY, rows=None, extra=0, lds=1):
    n = x.shape[0] if rows is None else len(rows)
    q = torch.full((n, ref.up(k, 16) + 16 * extra), 0x5A, dtype=torch.int8, device="cuda")
    s = torch.full((n, lds), -5.0, device="cuda")
    idx = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    g.int_quantize(x, qg.layout(dtype, x.shape[0], 2 * k if act == qg.MX_SWIGLU else k, ld=x.stride(0)), q,
                  qg.layout("i8", n, k, ld=q.stride(0)), s, qg.layout("f32", n, 1, ld=lds), act=act, rows=idx)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert (q[:, k:] == 0x5A).all() and (s[:, 1:] == -5.0).all(), "write past a row's end"
    return q[:, :k], s[:, 0]


def check(got, y):
    q, s = ref.quantise(y)
    assert np.array_equal(got[1], s, equal_nan=True), np.argwhere(got[1] != s)[:4].tolist()
    assert np.array_equal(got[0], q), (int((got[0] != q).sum()), np.argwhere(got[0] != q)[:4].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 16), (3, 31), (33, 64), (5, 100), (17, 257), (9, 500), (6, 1001), (3, 2047),
                                    (64, 4096), (33, 7201), (3, 14336), (2, 16392), (1, 65536)])
def test_identity(g, dtype, rows, k):
    x = sample(rows, k, dtype, rows * 7919 + k, spread=3)
    check(quantise(g, pitched(x, dtype, extra=rows & 1), dtype, k, extra=rows & 1, lds=1 + (rows & 3)), x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 64), (3, 33), (16, 1001), (7, 4096), (64, 2880), (40, 14336), (2, 20001), (1, 65536)])
def test_swiglu(g, dtype, rows, k):
    x = sample(rows, 2 * k, dtype, rows + 31 * k, spread=2)
    check(quantise(g, pitched(x, dtype), dtype, k, act=qg.MX_SWIGLU), ref.swiglu(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_ties_and_their_neighbours(g, dtype):
    """Scale 1 (largest 127): every half from 0.5 to 126.5 is a tie that goes to the even code, its neighbours are not."""
    halves = np.arange(127) + 0.5
    x = np.concatenate([[127.0], halves, halves * (1 + 2.0 ** -9), halves * (1 - 2.0 ** -9)])
    x = np.stack([x, -x, x * 2.0 ** -7, x * 0.75])
    x = torch.from_numpy(x).to(DT[dtype]).double().numpy()
    check(quantise(g, pitched(x, dtype), dtype, x.shape[1]), x)


def test_nearly_ties_in_fp32(g):
    """Values a step of fp32 on either side of (n + 1/2) scales, over scales of every mantissa pattern."""
    r = np.random.default_rng(3)
    amax = (1 + r.random(512)).astype(np.float32)
    s = (amax.astype(np.float64) / 127).astype(np.float32)
    n = r.integers(0, 126, (512, 96)) + 0.5
    v = (n * s[:, None].astype(np.float64)).astype(np.float32)
    v = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(9))], 1)
    v *= np.where(r.random(v.shape) < 0.5, -1, 1).astype(np.float32)
    x = np.concatenate([amax[:, None], v], 1).astype(np.float64)
    check(quantise(g, pitched(x, "f32"), "f32", x.shape[1]), x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", [qg.MX_IDENTITY, qg.MX_SWIGLU])
@pytest.mark.parametrize("k", [60, 700, 5000])
def test_nan_infinity_zero_and_tiny_rows(g, dtype, act, k):
    x = sample(9, k * (1 + act), dtype, 5)
    x[0, 3], x[1, 40], x[2, k - 1], x[3, x.shape[1] - 1] = np.nan, np.inf, -np.inf, np.nan
    x[4] = 0.0
    x[5] = -0.0
    x[6] *= 2.0 ** -20
    x[7] *= {"bf16": 2.0 ** -125, "f16": 2.0 ** -14, "f32": 2.0 ** -130}[dtype]
    x[8] *= {"bf16": 2.0 ** 124, "f16": 2.0 ** 12, "f32": 2.0 ** 124}[dtype]
    with np.errstate(over="ignore"):
        x = torch.from_numpy(x).to(DT[dtype]).double().numpy()
    x[8] = np.where(np.isfinite(x[8]), x[8], 1.0)
    check(quantise(g, pitched(x, dtype), dtype, k, act=act), ref.swiglu(x) if act else x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_of_far_gates(g, dtype):
    """Gates below -8, -32 and -88, beside ups so large that their products are the row's largest, or all there is."""
    k = 256
    x = sample(8, 2 * k, dtype, 9)
    gate = np.random.default_rng(2).uniform(-100, -1, (8, k))
    gate[1] = np.linspace(-33, -31, k)
    gate[2] = np.linspace(-9, -7, k)
    gate[3] = np.linspace(-104, -86, k)
    x[:, :k] = gate
    x[3, k:] *= 2.0 ** 100
    x[4, k:] *= 2.0 ** 60
    x[5, :k] = np.where(np.arange(k) % 7 == 0, gate[5], x[6, k:])
    x[6, :k], x[6, k:] = 2.0 ** -80, 2.0 ** -75
    x[7, :k], x[7, k:] = 2.0 ** 70, 2.0 ** 70  # past fp32
    x = torch.from_numpy(x).to(DT[dtype]).double().numpy()
    check(quantise(g, pitched(x, dtype), dtype, k, act=qg.MX_SWIGLU), ref.swiglu(x))


@pytest.mark.parametrize("act", [qg.MX_IDENTITY, qg.MX_SWIGLU])
@pytest.mark.parametrize("k", [72, 2100])
def test_gathered_rows(g, act, k):
    t = 9
    x = sample(t, k * (1 + act), "bf16", 11)
    rows = [3, 3, 0, 8, -1, 5, 9, 1 << 30, 7, 0, -(1 << 31)]
    y = np.array([x[r] if 0 <= r < t else np.zeros(x.shape[1]) for r in rows])
    check(quantise(g, pitched(x, "bf16"), "bf16", k, act=act, rows=rows), ref.swiglu(y) if act else y)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 33), (17, 4096), (300, 1001), (2000, 9000)])
def test_dequantise(g, dtype, rows, k):
    """The product of a code and a scale takes one rounding to the type, or one to fp32 (2^-24) before it."""
    r = np.random.default_rng(rows + k)
    q = r.integers(-128, 128, (rows, ref.up(k, 16))).astype(np.int8)
    s = (r.random((rows, 2)) + 0.5).astype(np.float32) * np.float32(2.0 ** -6)
    if rows > 2:
        s[1, 0], s[2, 0] = np.nan, 0.0
    y = torch.full((rows, ref.up(k, 16 // SIZE[dtype]) + 8), 3.0, dtype=DT[dtype], device="cuda")
    qt, st = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    g.int_dequantize(qt, qg.layout("i8", rows, k, ld=q.shape[1]), st, qg.layout("f32", rows, 1, ld=2), y,
                    qg.layout(dtype, rows, k, ld=y.stride(0)))
    want, got = q[:, :k].astype(np.float64) * s[:, :1].astype(np.float64), y[:, :k].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    tol = 2.0 ** -24 * np.abs(want)
    tol = np.nan_to_num(tol + ref.DT_EPS[dtype] * (np.abs(want) + tol) + ref.DT_TINY[dtype])
    assert (np.abs(np.nan_to_num(got) - np.nan_to_num(want)) <= tol).all()
    assert (y[:, k:] == 3.0).all()


def test_empty(g):
    x = torch.ones(4, 16, device="cuda", dtype=torch.bfloat16)
    s = torch.full((4,), -5.0, device="cuda")
    q = torch.zeros(4, 16, device="cuda", dtype=torch.int8)
    g.int_quantize(x, qg.layout("bf16", 4, 16), q, qg.layout("i8", 0, 16), s, qg.layout("f32", 0, 1))
    assert (s == -5.0).all()
    g.int_quantize(x, qg.layout("bf16", 4, 0, ld=16), q, qg.layout("i8", 4, 0, ld=16), s, qg.layout("f32", 4, 1))
    assert (s == 0).all() and not q.any()  # rows without columns: scale 0
    g.int_dequantize(q, qg.layout("i8", 4, 0, ld=16), s, qg.layout("f32", 4, 1), x, qg.layout("bf16", 4, 0, ld=16))
    assert (x == 1).all()


def test_rows_do_not_depend_on_their_neighbours(g):
    """A row's codes and scale are its own: alone, and among others, and called twice."""
    k = 3001
    x = sample(40, 2 * k, "f32", 21, spread=4)
    x[::3, :k] -= 40
    t = pitched(x, "f32")
    q, s = quantise(g, t, "f32", k, act=qg.MX_SWIGLU)
    for i in (0, 7, 39):
        q1, s1 = quantise(g, t[i:i + 1], "f32", k, act=qg.MX_SWIGLU)
        assert np.array_equal(q1[0], q[i]) and s1[0] == s[i]
