"""The choice of experts on the GPU against the definition in 64 bits: ids are equal. Weights: the scores' own errors in
fp32, 2^-23 each for exp2 and rcp, 0.61 |x| 2^-23 for the argument's rounding, up to 22 roundings of the sum, a division and a
product: (24 + 1.5 |x|) 2^-23 of the weight, |x| being how far the logit lies from the largest (softmax) or from zero."""
import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NINF = float("-inf")


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


def run(g, x, dtype, top_k, bias=None, sigmoid=False, extra=0, **kw):
    """x: float64 values of the type. Returns ids and weights, with what lies past them checked untouched."""
    t, e = x.shape
    per = 16 // SIZE[dtype]
    xt = torch.full((t, ref.up(e, per) + extra * per), 1e4, dtype=DT[dtype])
    xt[:, :e] = torch.from_numpy(x).to(DT[dtype])
    xt = xt.cuda()
    ids = torch.full((t, top_k + 3), -77, dtype=torch.int32, device="cuda")
    w = torch.full((t, top_k + 1), -77.0, device="cuda")
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    r = qg.routing(qg.ROUTE_SIGMOID if sigmoid else qg.ROUTE_SOFTMAX, top_k, **kw)
    g.route(r, xt, qg.layout(dtype, t, e, ld=xt.stride(0)), b, ids, qg.layout("i32", t, top_k, ld=top_k + 3), w,
            qg.layout("f32", t, top_k, ld=top_k + 1))
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert (ids[:, top_k:] == -77).all() and (w[:, top_k:] == -77).all(), "write past a row's end"
    return ids[:, :top_k], w[:, :top_k]


def check(g, x, dtype, top_k, bias=None, sigmoid=False, **kw):
    bias = None if bias is None else bias.astype(np.float32).astype(np.float64)
    ids, w = run(g, x, dtype, top_k, bias, sigmoid, **kw)
    kw.pop("extra", None)
    want, ww = ref.route(x, top_k, sigmoid, bias, **kw)
    assert np.array_equal(ids, want), np.argwhere(ids != want)[:4].tolist()
    far = np.where(np.isfinite(x), np.abs(x), 0).max() * (1 if sigmoid else 2)
    assert (np.abs(w - ww) <= (24 + 1.5 * min(far, 128)) * 2.0 ** -23 * np.abs(ww) + 2.0 ** -120).all()


def logits(t, e, dtype, seed, std=1.5):
    x = np.random.default_rng(seed).standard_normal((t, e)) * std
    return torch.from_numpy(x).to(DT[dtype]).double().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (5, 60, 4), (3, 64, 8), (130, 128, 6), (9, 160, 8), (7, 256, 8), (33, 384, 10),
                                   (6, 512, 32), (4, 777, 16), (3, 1024, 32), (2, 31, 31)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_plain(g, dtype, t, e, k, sigmoid):
    x = logits(t, e, dtype, t * 131 + e)
    check(g, x, dtype, k, sigmoid=sigmoid, renormalize=True, extra=t & 1)
    check(g, x, dtype, k, sigmoid=sigmoid, scale=2.5)
    bias = np.random.default_rng(e).standard_normal(e) * 0.1
    check(g, x, dtype, k, bias=bias, sigmoid=sigmoid, renormalize=True, scale=-1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("e,groups,top,k", [(16, 8, 4, 6), (256, 8, 4, 8), (160, 8, 3, 6), (64, 64, 9, 9), (72, 6, 2, 8), (96, 3, 2, 8),
                                            (512, 2, 1, 16), (1024, 4, 3, 10), (300, 5, 5, 4), (512, 16, 8, 22)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("best", [1, 2])
def test_groups(g, dtype, e, groups, top, k, sigmoid, best):
    x = logits(40, e, dtype, e + groups)
    x[3] = NINF
    x[4, : e // groups] = NINF
    x[5, 1:] = NINF
    x[6, e // groups:] = NINF
    bias = np.random.default_rng(e).standard_normal(e) * 0.2
    kw = dict(sigmoid=sigmoid, groups=groups, top_groups=top, group_best=best, renormalize=True)
    check(g, x, dtype, k, **kw)
    check(g, x, dtype, k, bias=bias, **kw)


MANY = 4099  # four tokens per wave, the last wave not full


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("e,k", [(1, 1), (8, 2), (31, 8), (64, 6), (100, 15), (256, 8), (500, 10)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_plain(g, dtype, e, k, sigmoid):
    x = logits(MANY, e, dtype, e)
    check(g, x, dtype, k, sigmoid=sigmoid, renormalize=True, extra=1)
    bias = np.random.default_rng(e).standard_normal(e) * 0.1
    check(g, x, dtype, k, bias=bias, sigmoid=sigmoid, scale=2.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("e,groups,top,k", [(256, 8, 4, 8), (160, 8, 3, 6), (72, 6, 2, 8), (96, 3, 2, 8), (512, 2, 1, 15), (48, 16, 5, 10),
                                            (64, 64, 9, 9)])
@pytest.mark.parametrize("sigmoid,best,biased", [(True, 2, True), (False, 1, True), (False, 2, False), (True, 1, False)])
def test_many_groups(g, dtype, e, groups, top, k, sigmoid, best, biased):
    x = logits(MANY, e, dtype, e + groups)
    x[3] = NINF
    x[4, : e // groups] = NINF
    x[5, 1:] = NINF
    x[4096, e // groups:] = NINF
    x[4097, ::2] = np.nan
    bias = np.random.default_rng(e).standard_normal(e) * 0.2 if biased else None
    check(g, x, dtype, k, bias=bias, sigmoid=sigmoid, groups=groups, top_groups=top, group_best=best, renormalize=True)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_in_doubt(g, sigmoid):
    """Most tokens' keys are too near for fp32, or equal: neighbours in a wave are redone one after the other."""
    r = np.random.default_rng(8)
    gap = 2.0 ** -22
    x = (1.0 + gap * r.permuted(np.tile(np.arange(96.0), (MANY, 1)), axis=1)).astype(np.float32).astype(np.float64)
    x[::3] = r.integers(-2, 3, (len(x[::3]), 96)) * 0.5
    x[5::7] = logits(len(x[5::7]), 96, "f32", 3)
    bias = (r.integers(0, 5, 96) * gap).astype(np.float32).astype(np.float64)
    check(g, x, "f32", 8, bias=bias, sigmoid=sigmoid)
    check(g, x, "f32", 8, bias=bias, sigmoid=sigmoid, groups=8, top_groups=2, group_best=2, renormalize=True)
    check(g, x, "f32", 8, sigmoid=sigmoid, groups=8, top_groups=2, group_best=2, renormalize=True)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_as_few(g, sigmoid, renorm):
    """The same rows in a large and a small call: the same ids, infinities and masks among them."""
    x = logits(MANY, 70, "f32", 2)
    x[0], x[1, 3:], x[2], x[3, ::2] = NINF, NINF, np.nan, np.nan
    x[4] = x[5] = -3.4028234663852886e38
    x[5, 40], x[6, [5, 9]], x[8] = 1.0, np.inf, 3.4028234663852886e38
    x[7, 0], x[7, 1:] = np.inf, NINF
    x[9] -= 200
    x[10] *= 60
    bias = np.random.default_rng(1).standard_normal(70)
    bias[[7, 9]], bias[11] = (NINF, np.inf), np.nan
    for b in (None, bias):
        with np.errstate(invalid="ignore"):
            check(g, x[:64], "f32", 8, bias=b, sigmoid=sigmoid, renormalize=renorm)
        ids, w = run(g, x, "f32", 8, b, sigmoid, renormalize=renorm)
        few, fw = run(g, x[:64], "f32", 8, b, sigmoid, renormalize=renorm)
        assert np.array_equal(ids[:64], few)
        assert (np.abs(w[:64] - fw) <= 2 * (24 + 1.5 * 128) * 2.0 ** -23 * np.abs(fw) + 2.0 ** -120).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
def test_ties_go_to_the_lowest_index(g, sigmoid, bias):
    r = np.random.default_rng(4)
    x = r.integers(-2, 3, (64, 200)) * 0.5
    x[0] = 0.0
    x[1] = np.where(np.arange(200) % 3 == 0, -0.0, 0.0)
    b = None if bias is None else np.full(200, bias)
    check(g, x, "f32", 8, bias=b, sigmoid=sigmoid, renormalize=True)
    check(g, x, "f32", 8, bias=b, sigmoid=sigmoid, renormalize=True, groups=8, top_groups=3, group_best=2)
    check(g, x, "f32", 8, bias=b, sigmoid=sigmoid, renormalize=True, groups=8, top_groups=3, group_best=1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("gap", [2.0 ** -18, 2.0 ** -21, 2.0 ** -23])
def test_keys_next_to_each_other(g, sigmoid, gap):
    """Logits and biases that fp32 scores cannot tell apart, and 64 bits can: the order of the sums, not of the logits."""
    r = np.random.default_rng(8)
    x = (1.0 + gap * r.permuted(np.tile(np.arange(96.0), (200, 1)), axis=1)).astype(np.float32).astype(np.float64)
    bias = (r.integers(0, 5, 96) * gap).astype(np.float32).astype(np.float64)
    check(g, x, "f32", 8, bias=bias, sigmoid=sigmoid)
    check(g, x, "f32", 8, bias=bias, sigmoid=sigmoid, groups=8, top_groups=2, group_best=2, renormalize=True)
    check(g, x, "f32", 8, sigmoid=sigmoid, groups=8, top_groups=2, group_best=2, renormalize=True)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_masks_infinities_and_nan(g, sigmoid, with_bias, renorm):
    x = logits(16, 70, "f32", 2)
    x[0] = NINF                                  # nothing left
    x[1, 3:] = NINF                              # fewer than top_k
    x[2] = np.nan
    x[3, ::2] = np.nan
    x[4] = -3.4028234663852886e38                # the type's lowest is a value, not a mask
    x[5] = -3.4028234663852886e38
    x[5, 40] = 1.0
    x[6, [5, 9]] = np.inf                        # share the softmax
    x[7, 0], x[7, 1:] = np.inf, NINF
    x[8] = 3.4028234663852886e38
    x[9] -= 200
    x[10] *= 60
    x[11, 17] = 80.0
    bias = np.random.default_rng(1).standard_normal(70)
    bias[[7, 9]] = NINF, np.inf
    bias[11] = np.nan
    with np.errstate(invalid="ignore"):
        check(g, x, "f32", 8, bias=bias if with_bias else None, sigmoid=sigmoid, renormalize=renorm)


def test_a_great_many_tokens(g):
    """Each row by itself against the rows of a smaller call: the ids are equal, the weights, summed in another order there, both
    within the bound above of the exact ones."""
    x = logits(512, 64, "f32", 77)
    ids, w = run(g, x, "f32", 4, renormalize=True)
    big = torch.from_numpy(x).float().cuda().repeat(9000, 1)  # 4.6 million rows
    t = big.shape[0]
    oi = torch.empty(t, 4, dtype=torch.int32, device="cuda")
    ow = torch.empty(t, 4, device="cuda")
    g.route(qg.routing(qg.ROUTE_SOFTMAX, 4, renormalize=True), big, qg.layout("f32", t, 64), None, oi, qg.layout("i32", t, 4), ow,
            qg.layout("f32", t, 4))
    assert torch.equal(oi, torch.from_numpy(ids).cuda().repeat(9000, 1))
    few = torch.from_numpy(w).cuda().repeat(9000, 1)
    assert ((ow - few).abs() <= 2 * (24 + 1.5 * 2 * np.abs(x).max()) * 2.0 ** -23 * few).all()


def test_no_tokens(g):
    ids, w = torch.full((1, 2), 9, dtype=torch.int32, device="cuda"), torch.full((1, 2), 9.0, device="cuda")
    x = torch.zeros(1, 8, device="cuda")
    g.route(qg.routing(top_k=2), x, qg.layout("f32", 0, 8), None, ids, qg.layout("i32", 0, 2), w, qg.layout("f32", 0, 2))
    assert (ids == 9).all() and (w == 9).all()


def test_tokens_past_2_to_the_32_threads(g):
    """2^28 tokens take 2^32 threads at 16 each: they go out in parts, and the last ones are written too."""
    t = (1 << 28) + 5
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free device memory")
    x = torch.zeros(t, 8, device="cuda", dtype=torch.bfloat16)
    x[:, 1] = 1
    x[-1, 0] = 2
    x[(1 << 27) - 1, 2], x[1 << 27, 3] = 3, 3
    ids = torch.full((t, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.empty(t, 1, device="cuda")
    g.route(qg.routing(qg.ROUTE_SOFTMAX, 1, renormalize=True), x, qg.layout("bf16", t, 5, ld=8), None, ids, qg.layout("i32", t, 1), w,
            qg.layout("f32", t, 1))
    ids = ids.flatten()
    assert ids[-1] == 0 and ids[(1 << 27) - 1] == 2 and ids[1 << 27] == 3
    assert int((ids == 1).sum()) == t - 3 and bool((w == 1).all())
