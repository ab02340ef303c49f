"""MXFP4 quantise and dequantise on the GPU against the definition in 64 bits. Codes and scales are compared for
equality: scaling by a power of two is exact, so each code is one rounding of an exactly known value."""
import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import mx_ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


def pitched(x, dtype, extra=0, fill=float("nan")):
    """Device tensor of x at a pitch of 16 bytes (plus `extra` chunks); the padding holds `fill`."""
    per = 16 // SIZE[dtype]
    t = torch.full((x.shape[0], mx_ref.up(x.shape[1], per) + extra * per), fill, dtype=DT[dtype])
    t[:, :x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    return t.cuda()


def quantise(g, x, dtype, k, act=qg.MX_IDENTITY, rows=None, extra=0):
    """Codes (rows x up(k, 32)) and scales of device tensor x, with what lies past them checked untouched."""
    n = x.shape[0] if rows is None else len(rows)
    nb = -(-k // 32)
    q = torch.full((n, nb * 16 + 16 * extra), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((n, mx_ref.up(nb, 16) + 16 * extra), 0x5A, dtype=torch.uint8, device="cuda")
    idx = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    g.mx_quantize(x, qg.layout(dtype, x.shape[0], 2 * k if act == qg.MX_SWIGLU else k, ld=x.stride(0)), q,
                  qg.layout("e2m1", n, k, ld=2 * q.stride(0)), s, qg.layout("e8m0", n, nb, ld=s.stride(0)), act=act, rows=idx)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert (q[:, nb * 16:] == 0x5A).all() and (s[:, nb:] == 0x5A).all(), "write past a row's end"
    return mx_ref.unpack(q[:, :nb * 16]), s[:, :nb]


def check(got, x, ignore_zero_sign=True):
    code, byte = mx_ref.quantise(x)
    assert np.array_equal(got[1], byte)
    a, b = got[0], code
    if ignore_zero_sign:  # a value that rounds to zero may carry either sign
        a, b = np.where(a == 8, 0, a), np.where(b == 8, 0, b)
    assert np.array_equal(a, b), (int((a != b).sum()), np.argwhere(a != b)[:4].tolist())


def sample(rows, cols, dtype, seed, spread=0.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * np.exp2(r.uniform(-spread, spread, (rows, cols)))
    return torch.from_numpy(x).to(DT[dtype]).double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 100), (17, 257), (64, 4096), (33, 7201), (301, 72)])
def test_identity(g, dtype, rows, k):
    x = sample(rows, k, dtype, rows * 7919 + k, spread=3)
    check(quantise(g, pitched(x, dtype, extra=rows & 1), dtype, k, extra=rows & 1), x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_border_at_every_scale(g, dtype):
    """A block per exponent: its maximum is 4 or 6 scales, the other values the borders themselves and their neighbours."""
    lo, hi = {"bf16": (-133, 127), "f16": (-24, 15), "f32": (-149, 127)}[dtype]
    rows = []
    for e in range(lo, hi + 1):
        for top in (4.0, 6.0, 7.5):
            v = [top]
            for b in mx_ref.BORDERS:
                for d in (-1, 0, 1):
                    v.append(b * (1 + d * 2.0 ** -7) * (-1) ** len(v))
            v += [5.0, -5.5, 0.0, 0.124, -0.126, 0.5, 1.0, 2.0, 3.0, 6.0]
            rows.append(np.ldexp(np.array(v[:32]), e - 2))
    with np.errstate(over="ignore"):
        x = np.array(rows)
        x = torch.from_numpy(x).to(DT[dtype]).double().numpy()
    x = np.where(np.isfinite(x), x, 0.0)
    check(quantise(g, pitched(x, dtype), dtype, 32), x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", [qg.MX_IDENTITY, qg.MX_SWIGLU])
def test_nan_infinity_and_zero_blocks(g, dtype, act):
    k = 160
    x = sample(4, k * (1 + act), dtype, 5)
    x[0, 3], x[1, 40], x[2, 70], x[3, 159] = np.nan, np.inf, -np.inf, np.nan
    x[:, 96:128] = 0.0
    if act:
        x[:, k + 96:k + 128] = -0.0
    check(quantise(g, pitched(x, dtype), dtype, k, act=act), mx_ref.swiglu(x) if act else x)


@pytest.mark.parametrize("act", [qg.MX_IDENTITY, qg.MX_SWIGLU])
def test_gathered_rows(g, act):
    k, t = 72, 9
    x = sample(t, k * (1 + act), "bf16", 11)
    rows = [3, 3, 0, 8, -1, 5, 9, 1 << 30, 7, 0, -(1 << 31)]
    y = np.array([x[r] if 0 <= r < t else np.zeros(x.shape[1]) for r in rows])
    check(quantise(g, pitched(x, "bf16"), "bf16", k, act=act, rows=rows), mx_ref.swiglu(y) if act else y)
    code, byte = quantise(g, pitched(x, "bf16"), "bf16", k, rows=[9, -1]) if not act else (np.zeros(1), np.zeros(1))
    assert not code.any() and not byte.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 64), (3, 33), (16, 1001), (7, 4096), (64, 2880)])
def test_swiglu(g, dtype, rows, k):
    x = sample(rows, 2 * k, dtype, rows + 31 * k, spread=2)
    check(quantise(g, pitched(x, dtype), dtype, k, act=qg.MX_SWIGLU), mx_ref.swiglu(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_swiglu_many_values(g, dtype):
    """8 million values: fp32 arithmetic alone would put several on the wrong side of a border."""
    x = sample(1024, 16384, dtype, 3, spread=1)
    check(quantise(g, pitched(x, dtype), dtype, 8192, act=qg.MX_SWIGLU), mx_ref.swiglu(x))


def test_swiglu_next_to_borders(g):
    """fp32 inputs whose product lies within one fp32 step of a border, or whose maximum lies so near a power of two."""
    r = np.random.default_rng(17)
    n = 2048
    gate = r.uniform(-4, 12, (n, 32)).astype(np.float32)
    silu = gate.astype(np.float64) / (1 + np.exp(-gate.astype(np.float64)))
    want = r.choice(mx_ref.BORDERS, (n, 32)) * r.choice([-1.0, 1.0], (n, 32))
    want[:, 5] = r.choice([4.0, 8.0, 6.0], n)
    up = (want / silu).astype(np.float32)
    up = np.where(r.random((n, 32)) < 0.5, np.nextafter(up, np.float32(0)), up)
    x = np.concatenate([gate, up], 1).astype(np.float64)
    check(quantise(g, pitched(x, "f32"), "f32", 32, act=qg.MX_SWIGLU), mx_ref.swiglu(x))


def test_swiglu_extremes(g):
    """Far negative gates, values beyond fp32's range either way, and blocks that underflow."""
    r = np.random.default_rng(23)
    x = np.zeros((8, 64), dtype=np.float32)
    x[0, :32], x[0, 32:] = r.uniform(-100, -20, 32), r.uniform(1, 2, 32)
    x[1, :32], x[1, 32:] = r.uniform(-90, -80, 32), r.uniform(1e30, 1e38, 32)
    x[2, :32], x[2, 32:] = r.uniform(1e19, 1e20, 32), r.uniform(1e19, 1e20, 32)  # past fp32's largest
    x[3, :32], x[3, 32:] = r.uniform(1e-20, 1e-19, 32), r.uniform(1e-20, 1e-19, 32)
    x[4, :32], x[4, 32:] = r.uniform(1e-30, 1e-28, 32), r.uniform(1e-30, 1e-28, 32)
    x[5, :32], x[5, 32:] = r.uniform(50, 200, 32), r.uniform(-1, 1, 32)
    x[6, :32], x[6, 32:] = -3e38, 3e38
    x[7, :32], x[7, 32:] = 3e38, r.uniform(-1, 1, 32)
    check(quantise(g, pitched(x.astype(np.float64), "f32"), "f32", 32, act=qg.MX_SWIGLU), mx_ref.swiglu(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (2, 31), (3, 33), (5, 100), (64, 4096), (9, 7201)])
def test_dequantise(g, dtype, rows, k):
    """Every code under random scales (0 and 255 among them), rounded once to the output's type."""
    r = np.random.default_rng(rows + k)
    nb = -(-k // 32)
    q = r.integers(0, 256, (rows, nb * 16), dtype=np.uint8)
    mid = {"f32": (0, 256), "bf16": (0, 256), "f16": (95, 145)}[dtype]
    s = np.full((rows, mx_ref.up(nb, 16)), 255, dtype=np.uint8)
    s[:, :nb] = r.integers(*mid, (rows, nb))
    s[0, 0] = 255 if rows > 1 else 120
    per = 16 // SIZE[dtype]
    y = torch.full((rows, mx_ref.up(k, per) + per), 7.0, dtype=DT[dtype], device="cuda")
    g.mx_dequantize(torch.from_numpy(q).cuda(), qg.layout("e2m1", rows, k), torch.from_numpy(s).cuda(),
                    qg.layout("e8m0", rows, nb), y, qg.layout(dtype, rows, k, ld=y.stride(0)))
    y = y.cpu()
    assert (y[:, k:] == 7.0).all()
    ref = torch.from_numpy(mx_ref.values(mx_ref.unpack(q), s[:, :nb])[:, :k])
    assert torch.equal(torch.nan_to_num(y[:, :k].double(), 1.5e300, 3e300, -3e300),
                       torch.nan_to_num(ref.to(DT[dtype]).double(), 1.5e300, 3e300, -3e300))


def test_dequantise_bytes_0_to_254_exactly_in_fp32(g):
    s = np.arange(256, dtype=np.uint8).reshape(1, 256)
    q = np.tile(mx_ref.pack(np.arange(32, dtype=np.uint8).reshape(1, 32) % 16), (1, 256))
    y = torch.empty(1, 8192, device="cuda")
    g.mx_dequantize(torch.from_numpy(q).cuda(), qg.layout("e2m1", 1, 8192), torch.from_numpy(s).cuda(),
                    qg.layout("e8m0", 1, 256), y, qg.layout("f32", 1, 8192))
    with np.errstate(over="ignore"):
        ref = mx_ref.values(mx_ref.unpack(q), s).astype(np.float32)
    y = y.cpu().numpy()
    assert np.array_equal(y, ref, equal_nan=True)


def test_stream_and_graph(g):
    """On a stream of its own, and captured: replays agree with the eager result, with eager work between them."""
    x = sample(40, 192, "bf16", 2)
    xd = pitched(x, "bf16")
    q = torch.zeros(40, 48, dtype=torch.uint8, device="cuda")
    s = torch.zeros(40, 16, dtype=torch.uint8, device="cuda")
    y = torch.zeros(40, 96, dtype=torch.bfloat16, device="cuda")
    ld = (qg.layout("bf16", 40, 192), qg.layout("e2m1", 40, 96), qg.layout("e8m0", 40, 3), qg.layout("bf16", 40, 96))

    def both():
        g.mx_quantize(xd, ld[0], q, ld[1], s, ld[2], act=qg.MX_SWIGLU)
        g.mx_dequantize(q, ld[1], s, ld[2], y, ld[3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    want = mx_ref.values(*mx_ref.quantise(mx_ref.swiglu(x)))
    assert np.array_equal(y.double().cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(3):
        x = sample(40, 192, "bf16", 20 + i)
        xd.copy_(pitched(x, "bf16"))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(y.double().cpu().numpy(), mx_ref.values(*mx_ref.quantise(mx_ref.swiglu(x))))


def test_more_units_than_32_bits_count(g):
    """2^32 units of 8 elements and more: 4.2 million rows of 8192, gathered from 16; codes, scales and values whole."""
    k, n, t = 8192, (1 << 22) + 3001, 16
    x = sample(t, k, "bf16", 4)
    code, byte = mx_ref.quantise(x)
    rows = torch.randint(0, t, (n,), device="cuda", dtype=torch.int32)
    q = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(n, k // 32, dtype=torch.uint8, device="cuda")
    y = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    qd, sd = qg.layout("e2m1", n, k), qg.layout("e8m0", n, k // 32)
    g.mx_quantize(pitched(x, "bf16"), qg.layout("bf16", t, k), q, qd, s, sd, rows=rows)
    g.mx_dequantize(q, qd, s, sd, y, qg.layout("bf16", n, k))
    values = torch.from_numpy(mx_ref.values(code, byte)).to(torch.bfloat16).cuda()
    code, byte = torch.from_numpy(mx_ref.pack(code)).cuda(), torch.from_numpy(byte).cuda()
    step = 1 << 18
    for i in range(0, n, step):
        r = rows[i:i + step].long()
        assert torch.equal(s[i:i + step], byte[r])
        assert torch.equal(y[i:i + step], values[r])
        got, want = q[i:i + step], code[r]  # a code of zero may carry either sign
        for nibble in (15, 240):
            a, b = got & nibble, want & nibble
            assert bool(((a == b) | ((a | b) & (nibble & 119) == 0)).all())
    del q, s, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act,n", [(qg.MX_SWIGLU, (1 << 16) + 5), (qg.MX_IDENTITY, (1 << 17) + 5)])
def test_more_threads_than_one_launch_holds(g, act, n):
    """A grid of 2^32 threads and more (two units to a thread gated, four plain): rows of 2^20, gathered from 3; every
    byte of the codes and scales."""
    k, t = 1 << 20, 3
    x = sample(t, k * (1 + act), "bf16", 6)
    xd = pitched(x, "bf16")
    rows = torch.randint(0, t, (n,), device="cuda", dtype=torch.int32)
    q = torch.full((n, k // 2), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((n, k // 32), 0x5A, dtype=torch.uint8, device="cuda")
    g.mx_quantize(xd, qg.layout("bf16", t, k * (1 + act)), q, qg.layout("e2m1", n, k), s, qg.layout("e8m0", n, k // 32), act=act,
                  rows=rows)
    few = quantise(g, xd, "bf16", k, act=act)
    check(few, mx_ref.swiglu(x) if act else x)
    code, byte = torch.from_numpy(mx_ref.pack(few[0])).cuda(), torch.from_numpy(few[1]).cuda()
    step = 1 << 12
    for i in range(0, n, step):
        r = rows[i:i + step].long()
        assert torch.equal(s[i:i + step], byte[r]), i
        assert torch.equal(q[i:i + step], code[r]), i
    del q, s
    torch.cuda.empty_cache()


def test_swiglu_subnormal_gates(g):
    """fp32 gates of a few bits against ups that bring the product far above fp32's smallest: g / (1 + exp(-g)) must not
    be rounded to the subnormal grid on the way."""
    r = np.random.default_rng(29)
    n = 1024
    at, by = r.integers(-149, -126, (n, 1)), r.integers(90, 121, (n, 1))
    gate = np.ldexp(r.uniform(1, 8, (n, 32)) * r.choice([-1.0, 1.0], (n, 32)), at).astype(np.float32)
    up = np.ldexp(r.uniform(1, 4, (n, 32)), by).astype(np.float32)
    x = np.concatenate([gate, up], 1).astype(np.float64)
    check(quantise(g, pitched(x, "f32"), "f32", 32, act=qg.MX_SWIGLU), mx_ref.swiglu(x), ignore_zero_sign=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_swiglu_bytes_do_not_depend_on_the_neighbours(g, dtype):
    """A row's bytes, the sign of its zeros among them, are those of the row alone, whether or not other rows need 64 bits."""
    k = 32
    x = sample(64, 2 * k, dtype, 31, spread=1)
    x[::2, 0:8] = 0.0
    x[::2, 8:16] = -0.0
    x[::4, k + 16:k + 24] = 0.0
    x[1::2, 3] = -40.0
    whole = quantise(g, pitched(x, dtype), dtype, k, act=qg.MX_SWIGLU)
    check(whole, mx_ref.swiglu(x), ignore_zero_sign=False)
    for i in range(0, 64, 2):
        code, byte = quantise(g, pitched(x[i:i + 1], dtype), dtype, k, act=qg.MX_SWIGLU)
        assert np.array_equal(code[0], whole[0][i]) and np.array_equal(byte[0], whole[1][i])
