"""The choice with a bias where the keys on both sides of the cut lie within their fp32 errors, and these errors differ: the ids
are those of 64 bits (checked as in the tests of the choice). A strong logit with a negative bias has an fp32 key off by some 2^-25,
a weak one's key is off by 2^-28: the one behind the first that is left out may be the better one."""
import numpy as np
import pytest

import quantized_gemm_bf16_amd as qg
from tests.test_gpu_route import MANY, check, logits

pytestmark = pytest.mark.gpu
FEW = 300  # a token per wave


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


def f32(x):
    return np.asarray(x, np.float32).astype(np.float64)


def mixed(t, top_k, gap, sigmoid, seed):
    """24 weak logits whose keys are their biases, `gap` apart, and strong logits of negative bias whose keys come to lie around the
    top_k-th of those, a last bit of the logit at a time."""
    r = np.random.default_rng(seed)
    e, weak = 64, 24
    at = r.permutation(e)
    bias, x = np.full(e, -2.0), np.full((t, e), -30.0)
    bias[at[:weak]] = 0.11 - gap * np.arange(weak)
    cut = 0.11 - gap * (top_k - 0.5)
    strong = at[weak:weak + 6]
    for i, j in enumerate(strong):
        bias[j] = -0.8636 + 0.0101 * i
    bias = f32(bias)
    # sigmoid(l) + bias = cut: in a softmax by one other logit of -l below the strong one of 0
    l = -np.log(1.0 / (cut - bias[strong]) - 1.0)
    l = f32(l + 2.0 ** -22 * r.integers(-60, 61, (t, len(strong))))
    if sigmoid:
        x[:, strong] = l
    else:  # one of the strong ones each
        i, which = np.arange(t), r.integers(0, len(strong), t)
        x[i, strong[which]] = 0.0
        x[:, at[-1]] = -l[i, which]
    return x, bias


def test_example(g):
    """Keys in fp32 0.1100000516, 0.1100000218, 0.1100000143; the third is 0.1100000576."""
    x = np.array([[-30.0, -30.0, float.fromhex("0x1.ced7c8p+1")]])
    bias = np.array([float.fromhex(b) for b in ("0x1.c28f6ap-4", "0x1.c28f62p-4", "-0x1.ba45b4p-1")])
    for t in (1, MANY):
        check(g, np.repeat(x, t, 0), "f32", 1, bias=bias, sigmoid=True)


@pytest.mark.parametrize("t", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("top_k", [1, 2, 8, 15])
@pytest.mark.parametrize("gap", [2.0 ** -25, 2.0 ** -24, 2.0 ** -22, 2.0 ** -20])
def test_errors_of_different_size(g, t, sigmoid, top_k, gap):
    x, bias = mixed(t, top_k, gap, sigmoid, top_k)
    check(g, x, "f32", top_k, bias=bias, sigmoid=sigmoid)


@pytest.mark.parametrize("t", [FEW, MANY])
@pytest.mark.parametrize("bias", [0.0, 0.25])
@pytest.mark.parametrize("top_k", [1, 2, 5, 15])
def test_equal_experts_on_both_sides_of_the_cut(g, t, bias, top_k):
    """Scores of a sigmoid that fp32 rounds to 1: top_k + 1 or more equal experts, then better ones of higher index."""
    r = np.random.default_rng(top_k)
    x = logits(t, 40, "bf16", top_k)
    for row in x:
        at = np.sort(r.permutation(40)[:top_k + 1 + r.integers(1, 9)])
        row[at] = 20.0
        row[at[top_k + 1:]] = r.integers(20, 23, len(at) - top_k - 1)
    x[0] = 0.0
    x[0, [3, 8, 30]] = 20.0, 20.0, 21.0
    check(g, x, "f32", top_k, bias=np.full(40, bias), sigmoid=True)
    check(g, x, "bf16", top_k, bias=np.full(40, bias), sigmoid=True, renormalize=True)
    check(g, x, "f32", top_k, bias=np.full(40, bias), sigmoid=True, groups=5, top_groups=4, group_best=1)


@pytest.mark.parametrize("t", [FEW, MANY])
@pytest.mark.parametrize("top_k", [2, 3, 5, 15])
def test_equal_small_scores_of_a_softmax(g, t, top_k):
    """One logit takes the softmax; the others' scores vanish beside a bias that all have, the equal ones' at the cut too."""
    r = np.random.default_rng(top_k)
    x = np.full((t, 40), -9.0)
    for row in x:
        at = np.sort(r.permutation(40)[:top_k + 1 + r.integers(1, 9)])
        row[at[top_k:]] = r.integers(-9, -6, len(at) - top_k)
        row[at[0]] = 30.0
    check(g, x, "f32", top_k, bias=np.full(40, 0.25))
    check(g, x, "bf16", top_k, bias=np.full(40, 0.25), renormalize=True)


@pytest.mark.parametrize("t", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_equal_pairs_at_the_cut(g, t, sigmoid):
    """Whole numbers and halves: pairs at the cut with nothing near them, with a third equal one, and with nothing behind them."""
    r = np.random.default_rng(3)
    x = r.integers(-8, 9, (t, 24)) * 0.5
    x[::3, 9:] = -np.inf
    for k in (1, 4, 8, 9, 15):
        check(g, x, "f32", k, bias=np.zeros(24), sigmoid=sigmoid)
        check(g, x, "f32", k, bias=f32(np.arange(24) % 3 * 0.125), sigmoid=sigmoid)
