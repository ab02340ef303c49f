"""int8 products with scales per token and channel over experts and over batches. The sum of codes is exact; the fp32 value
acc U V alpha takes four roundings (the sum's conversion among them), beta C one more, the result half a step of its type."""
import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


@pytest.fixture(scope="module")
def ws():
    return qg.workspace()


def kernels():
    return [i for i, n in enumerate(qg.kernel_names()) if "_I8_" in n]


class Problem:
    """counts: rows of each group. The padding past K holds extreme codes of opposite signs in A and B."""

    def __init__(self, counts, n, k, out="bf16", batched=False, shared=False, c=None, seed=0, ldu=1, ldv=1, behind=0):
        r = np.random.default_rng(seed)
        self.counts, self.n, self.k, self.out, self.batched = counts, n, k, out, batched
        e, m = len(counts), int(sum(counts)) + behind
        self.e, self.m = e, m
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        pitch = ref.up(k, 16) + 16
        nb = 1 if shared else e
        self.A = np.full((m, pitch), 127, np.int8)
        self.B = np.full((nb, n, pitch), -128, np.int8)
        self.A[:, :k] = r.integers(-128, 128, (m, k))
        self.B[..., :k] = r.integers(-128, 128, (nb, n, k))
        self.U = r.uniform(0.001, 0.01, (m, ldu)).astype(np.float32)
        self.V = r.uniform(0.001, 0.01, (nb, n, ldv)).astype(np.float32)
        self.c = c
        pn = ref.up(n, 16)
        self.C = torch.from_numpy(r.standard_normal((m, pn))).to(DT[c]) if c else None
        self.t = [torch.from_numpy(x).cuda() for x in (self.A, self.B, self.U, self.V)]
        self.offt = torch.from_numpy(self.off).cuda()
        self.Ct = self.C.cuda() if c else None
        self.D = torch.full((m, pn), -77.0, dtype=torch.int8 if out == "i8" else DT[out], device="cuda")
        kw = dict(num=e) if batched else dict(num=e, offsets=self.offt.data_ptr())
        rows = counts[0] if batched else m
        lay = lambda t, cols, ld: qg.layout(t, rows, cols, ld=ld, **kw, stride=rows * ld if batched else 0)  # noqa: E731
        self.Ad, self.Ud, self.Dd = lay("i8", k, pitch), lay("f32", 1, ldu), lay(out, n, pn)
        self.Cd = lay(c, n, pn) if c else None
        self.Bd = qg.layout("i8", n, k, ld=pitch, num=e, stride=0 if shared else n * pitch)
        self.Vd = qg.layout("f32", n, 1, ld=ldv, num=e, stride=0 if shared else n * ldv)

    def op(self, **kw):
        return qg.operation(quant_a=W8A8, quant_b=W8A8, **kw)

    def run(self, g, ws, alpha=1.0, beta=0.0, op=None):
        A, B, U, V = self.t
        self.D.fill_(-77)
        g.run(op or self.op(), alpha, A, self.Ad, U, self.Ud, B, self.Bd, V, self.Vd, beta, self.Ct, self.Cd, self.D, self.Dd, ws.desc)
        d = self.D.double().cpu().numpy()
        end = self.off[-1]
        assert (d[:, self.n:] == -77).all() and (d[end:] == -77).all(), "write past column N or behind the last group"
        return d[:end, :self.n]

    def exact(self, alpha=1.0, beta=0.0):
        out = []
        for e in range(self.e):
            q = 0 if len(self.B) == 1 else e
            rows = slice(self.off[e], self.off[e + 1])
            acc = self.A[rows, :self.k].astype(np.float64) @ self.B[q, :, :self.k].astype(np.float64).T
            out.append(acc * self.U[rows, :1].astype(np.float64) * self.V[q, :, 0].astype(np.float64))
        x = np.concatenate(out) * alpha
        tol = 2.0 ** -24 * 4.01 * np.abs(x)
        if beta:
            x = x + beta * self.C[:self.off[-1], :self.n].double().numpy()
            tol = tol + 2.0 ** -24 * 1.01 * np.abs(x)
        return x, tol

    def check(self, g, ws, alpha=1.0, beta=0.0, op=None):
        d = self.run(g, ws, alpha, beta, op)
        x, tol = self.exact(alpha, beta)
        tol = tol + ref.DT_EPS[self.out] * (np.abs(x) + tol) + ref.DT_TINY[self.out]
        assert (np.abs(d - x) <= tol).all(), np.argwhere(np.abs(d - x) > tol)[:4].tolist()
        return d


COUNTS = {"ragged": [0, 3, 1, 40, 0, 300, 17, 129, 0], "one": [5], "decode": [2, 1, 3, 0, 2, 1, 4, 3] * 4, "empty": [0, 0, 0]}


@pytest.mark.parametrize("kernel", [None] + kernels())
@pytest.mark.parametrize("counts", ["ragged", "one", "decode"])
@pytest.mark.parametrize("n,k", [(300, 528), (72, 1001), (17, 5)])
def test_experts(g, ws, kernel, counts, n, k):
    p = Problem(COUNTS[counts], n, k, "bf16", seed=n, behind=5)
    p.check(g, ws, op=None if kernel is None else p.op(policy=qg.POLICY_FORCE, kernel=kernel))


@pytest.mark.parametrize("kernel", [None] + kernels())
@pytest.mark.parametrize("out,c", [("f32", None), ("f16", "f16"), ("bf16", "f32"), ("f32", "bf16")])
def test_types_alpha_beta_and_strides(g, ws, kernel, out, c):
    p = Problem([60, 0, 200, 1], 200, 300, out, c=c, seed=7, ldu=3, ldv=2)
    p.check(g, ws, 0.75, -0.5 if c else 0.0, op=None if kernel is None else p.op(policy=qg.POLICY_FORCE, kernel=kernel))


@pytest.mark.parametrize("rows", [1, 16, 40, 300])
@pytest.mark.parametrize("shared", [False, True])
def test_batches(g, ws, rows, shared):
    p = Problem([rows] * 5, 136, 272, "bf16", batched=True, shared=shared, c="bf16", seed=rows, ldu=2)
    p.check(g, ws, 1.0, 1.0)


def test_experts_that_share_weights(g, ws):
    Problem([30, 0, 70], 100, 200, "f32", shared=True, seed=3).check(g, ws)


def test_nothing_to_do(g, ws):
    Problem(COUNTS["empty"], 64, 64, behind=3).run(g, ws)
    p = Problem([3, 4], 64, 0)  # K of zero: zeros
    assert not p.run(g, ws).any()


def test_epilogue(g, ws):
    """bias, ReLU, and int8 codes: the code is off by one at most where the scaled value is next to a half."""
    p = Problem([100, 30], 128, 256, "f32", seed=5)
    bias = torch.linspace(-1, 1, 128, device="cuda")
    x, tol = p.exact()
    d = p.run(g, ws, op=p.op(epilogue=qg.EPI_BIAS | qg.EPI_RELU, bias=bias))
    want = np.maximum(x + bias.double().cpu().numpy(), 0)
    assert (np.abs(d - want) <= tol + 2.0 ** -24 * (np.abs(want) + tol) * 2).all()
    p = Problem([100, 30], 128, 256, "i8", seed=5)
    scale = torch.rand(130, device="cuda") * 50
    d = p.run(g, ws, op=p.op(epilogue=qg.EPI_QUANT_I8, row_scale=scale, zero_point=3.0))
    t = x * scale.double().cpu().numpy()[:, None] + 3.0
    off = tol * scale.double().cpu().numpy()[:, None] + 2.0 ** -24 * (np.abs(t) + 3)
    assert ((d >= np.clip(np.rint(t - off), -128, 127)) & (d <= np.clip(np.rint(t + off), -128, 127))).all()


@pytest.mark.parametrize("counts,n,k", [([900, 30, 0, 1200, 5, 700], 2000, 1500), ([1] * 64 + [0] * 20, 2048, 2080)])
def test_larger(g, ws, counts, n, k):
    p = Problem(counts, n, k, "bf16", seed=11)
    d = p.check(g, ws)
    assert np.array_equal(d, p.run(g, ws))


def test_no_alloc_gives_the_same(g, ws):
    p = Problem([5, 0, 30], 96, 400, "f32", seed=1)
    d = p.run(g, ws)
    A, B, U, V = p.t
    p.D.fill_(-77)
    assert g.run_noalloc_raw(p.op(), 1.0, A, p.Ad, U, p.Ud, B, p.Bd, V, p.Vd, 0.0, None, None, p.D, p.Dd) == qg.OK
    assert np.array_equal(p.D.double().cpu().numpy()[:35, :96], d)
