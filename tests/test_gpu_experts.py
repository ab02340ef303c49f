"""Sorting choices by expert (equal to the definition) and putting results together on the GPU. A combined value is off by
K + 1 roundings of fp32 sums and products, each at most 2^-24 of sum |w r| + |beta c|, and half a step of its type."""
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


@pytest.fixture(scope="module")
def ws():
    return qg.workspace()


def group(g, ids, experts, ws=None, extra=0):
    t, k = ids.shape
    it = torch.full((t, k + extra), 0, dtype=torch.int32)
    it[:, :k] = torch.from_numpy(ids)
    it = it.cuda()
    off = torch.full((experts + 2,), -77, dtype=torch.int32, device="cuda")
    rows, back = (torch.full((t * k + 1,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    g.group_rows(experts, it, qg.layout("i32", t, k, ld=k + extra), off, rows, back, ws.desc if ws else None)
    off, rows, back = off.cpu().numpy(), rows.cpu().numpy(), back.cpu().numpy()
    assert off[-1] == -77 and rows[-1] == -77 and back[-1] == -77, "write past the end"
    return off[:-1], rows[:-1], back[:-1].reshape(t, k)


@pytest.mark.parametrize("t,k,experts", [(1, 1, 1), (1, 8, 64), (16, 8, 64), (63, 3, 5), (64, 1, 2), (65, 1, 1023), (500, 8, 256),
                                         (1000, 8, 60), (1024, 8, 8), (1025, 8, 64), (3001, 7, 129), (20000, 8, 256), (70000, 2, 1023)])
@pytest.mark.parametrize("drop", [False, True])
def test_group(g, ws, t, k, experts, drop):
    r = np.random.default_rng(t + k)
    ids = r.integers(0, experts, (t, k)).astype(np.int32)
    if drop:
        ids = np.where(r.random((t, k)) < 0.4, r.choice([-1, experts, 1 << 30, -(1 << 31)], (t, k)), ids).astype(np.int32)
    got = group(g, ids, experts, ws, extra=t % 3)
    for a, b in zip(got, ref.group(ids, experts)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("t", [200, 9000])
def test_group_of_one_kind(g, ws, t):
    for fill in (0, 16, -1, 17):  # all the first expert's, all the last one's, nobody's
        ids = np.full((t, 3), fill, np.int32)
        for a, b in zip(group(g, ids, 17, ws), ref.group(ids, 17)):
            assert np.array_equal(a, b)


def test_group_of_nothing(g):
    off = torch.full((9,), -77, dtype=torch.int32, device="cuda")
    g.group_rows(8, None, qg.layout("i32", 0, 4), off, None, None)
    assert (off == 0).all()


def test_group_without_a_workspace(g):
    ids = np.arange(8192, dtype=np.int32).reshape(1024, 8) % 77
    for a, b in zip(group(g, ids, 77), ref.group(ids, 77)):
        assert np.array_equal(a, b)
    it = torch.zeros(1025, 8, dtype=torch.int32, device="cuda")
    off, rows, back = (torch.zeros(9000, dtype=torch.int32, device="cuda") for _ in range(3))
    assert g.group_rows_raw(77, it, qg.layout("i32", 1025, 8), off, rows, back) == qg.ERR_WORKSPACE


def combine(g, r, back, w, out, c=None, beta=0.0, extra=0, dtype="bf16", c_type="f32"):
    """r (float64 values of `dtype`), back, w (float32), c. Returns Y as float64 and its exact value with the bound."""
    def pitched(x, t):
        per = 16 // SIZE[t]
        p = torch.full((x.shape[0], ref.up(x.shape[1], per) + extra * per), float("nan"), dtype=DT[t])
        p[:, :x.shape[1]] = torch.from_numpy(x)
        return p.cuda()

    (n, h), (t, k) = r.shape, back.shape
    rt = pitched(r, dtype)
    y = torch.full((t, ref.up(h, 16 // SIZE[out]) + 8), -77.0, dtype=DT[out], device="cuda")
    wt = torch.full((t, k + 2), float("nan"))
    wt[:, :k] = torch.from_numpy(w)
    wt, bt = wt.cuda(), torch.from_numpy(back).cuda()
    ct = pitched(c, c_type) if c is not None else None
    g.combine(rt, qg.layout(dtype, n, h, ld=rt.stride(0)), bt, wt, qg.layout("f32", t, k, ld=k + 2), y, qg.layout(out, t, h, ld=y.stride(0)),
              beta=beta, C=ct, Cd=qg.layout(c_type, t, h, ld=ct.stride(0)) if c is not None else None)
    assert (y[:, h:] == -77).all(), "write past a row's end"
    there = (back >= 0) & (back < n)
    part = np.where(there, w, 0.0).astype(np.float64)[..., None] * r[np.clip(back, 0, max(n - 1, 0))] if n else np.zeros((t, k, h))
    part = np.where(there[..., None], part, 0.0)
    want, size = part.sum(1), np.abs(part).sum(1)
    if c is not None:
        want, size = want + beta * c, size + np.abs(beta * c)
    tol = (k + 1) * 2.0 ** -24 * size
    return y[:, :h].double().cpu().numpy(), want, tol + ref.DT_EPS[out] * (np.abs(want) + tol) + ref.DT_TINY[out]


def values(shape, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).to(DT[dtype]).double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,k,h", [(1, 1, 1), (1, 8, 7168), (3, 2, 33), (130, 6, 200), (17, 8, 4096), (5, 19, 1001), (300, 4, 72)])
def test_combine(g, dtype, out, t, k, h):
    r = np.random.default_rng(t + h)
    n = t * k
    back = r.permutation(n).astype(np.int32).reshape(t, k)
    if t > 2:
        back = np.where(r.random((t, k)) < 0.3, r.choice([-1, n, 1 << 30, -(1 << 31)], (t, k)), back).astype(np.int32)
        back[1] = -1
    w = r.random((t, k)).astype(np.float32)
    c_type = {"bf16": "f32", "f16": "bf16", "f32": "f16"}[out]
    for c, beta in ((None, 0.0), (values((t, h), c_type, 3), 1.0), (values((t, h), c_type, 4), -0.5)):
        y, want, tol = combine(g, values((n, h), dtype, 5), back, w, out, c, beta, extra=t & 1, dtype=dtype, c_type=c_type)
        assert (np.abs(y - want) <= tol).all()


def test_combine_skips_what_is_not_there(g):
    """Rows and weights of choices that are nobody's are not read into the sum, whatever they hold."""
    r = values((4, 64), "bf16", 1)
    r[3] = np.nan
    back = np.array([[0, -1], [-1, -1], [2, 4]], np.int32)
    w = np.array([[0.5, np.nan], [np.inf, np.nan], [1.0, np.inf]], np.float32)
    w64 = np.where((back >= 0) & (back < 4), w, 0.0).astype(np.float32)
    y, _, _ = combine(g, r, back, w, "f32")
    _, want, tol = combine(g, np.nan_to_num(r), back, w64, "f32")
    assert (np.abs(y - want) <= tol).all() and not y[1].any()


def test_combine_without_choices_or_rows(g):
    c = values((5, 24), "f32", 2)
    y, want, tol = combine(g, np.zeros((0, 24)), np.zeros((5, 0), np.int32), np.zeros((5, 0), np.float32), "f32", c, 2.0)
    assert np.array_equal(y, 2.0 * c)
    y, want, tol = combine(g, np.zeros((0, 24)), np.zeros((5, 2), np.int32), np.ones((5, 2), np.float32), "bf16")
    assert not y.any()


def test_combine_in_place(g):
    """Y may be C: the residual is added to where it stands."""
    t, k, h = 37, 4, 520
    r = values((t * k, h), "bf16", 6)
    back = np.random.default_rng(1).permutation(t * k).astype(np.int32).reshape(t, k)
    w = np.random.default_rng(2).random((t, k)).astype(np.float32)
    c = torch.randn(t, h, device="cuda", dtype=torch.bfloat16)
    y = torch.empty_like(c)
    rt, bt, wt = torch.from_numpy(r).to(torch.bfloat16).cuda(), torch.from_numpy(back).cuda(), torch.from_numpy(w).cuda()
    d = qg.layout("bf16", t, h)
    for to in (y, c):
        g.combine(rt, qg.layout("bf16", t * k, h), bt, wt, qg.layout("f32", t, k), to, d, beta=1.0, C=c, Cd=d)
    assert torch.equal(c, y)
