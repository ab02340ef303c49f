"""MXFP4 products on the GPU against the definition in 64 bits.

Products of two values are exact in fp32 and the hardware's and the engine's sums are fp32, so an output is off by
at most the rounding of its own type (half a step) and of K - 1 fp32 additions, each half a step of a partial sum that
is at most absdot = sum |a b|: 2^-24 (K + 2) absdot bounds these whatever their order, and alpha, beta c and their sum
add 2^-23 (|alpha| absdot + |beta c|)."""
import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import mx_ref

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
MX = (qg.QUANT_MX, 32, 1, 0)


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


@pytest.fixture(scope="module")
def ws():
    return qg.workspace()


def stored(rows, k, r, extra=0, spread=4):
    """Random codes and scales as stored: the padding (codes past K, scales past the last block) holds 6s and NaN."""
    nb = -(-k // 32)
    code = np.full((rows, nb * 32 + 32 * extra), 7, dtype=np.uint8)
    code[:, :k] = r.integers(0, 16, (rows, k))
    s = np.full((rows, mx_ref.up(nb, 16) + 16 * extra), 255, dtype=np.uint8)
    s[:, :nb] = 127 + r.integers(-spread, spread + 1, (rows, nb))
    val = mx_ref.values(code[:, :nb * 32], s[:, :nb])[:, :k]
    return torch.from_numpy(mx_ref.pack(code)).cuda(), torch.from_numpy(s).cuda(), val


class Problem:
    def __init__(self, m, n, k, out="bf16", seed=0, counts=None, c=None, extra=0, share=False, batched=0):
        r = np.random.default_rng(seed)
        self.m, self.n, self.k, self.out, self.counts = m, n, k, out, counts
        nb = -(-k // 32)
        e = len(counts) if counts is not None else batched
        self.a, self.sa, self.av = stored(max(1, batched) * m, k, r, extra)
        self.b, self.sb, self.bv = stored((1 if share else max(1, e)) * n, k, r, extra)
        lk, ls = self.a.stride(0) * 2, self.sa.stride(0)
        self.ldn = mx_ref.up(n, 16) + 16 * extra
        rows = self.a.shape[0]
        self.d = torch.full((rows, self.ldn), -7 if out == "i8" else float("nan"), dtype=TORCH[out], device="cuda")
        off = 0
        if counts is not None:
            self.off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
            off = self.off.data_ptr()
        bs, vs = (0, 0) if share or not e else (n * lk, n * ls)

        def rowwise(t, cols, ld):
            return qg.layout(t, m, cols, ld=ld, num=e, offsets=off, stride=m * ld if batched else 0)

        self.c = self.cv = self.cd = None
        if c:
            cv = torch.from_numpy(r.standard_normal((rows, self.ldn)) * 30).to(TORCH[c])
            self.c, self.cv = cv.cuda(), cv.double().numpy()[:, :n]
            self.cd = rowwise(c, n, self.ldn)
        self.ad, self.ud, self.dd = rowwise("e2m1", k, lk), rowwise("e8m0", nb, ls), rowwise(out, n, self.ldn)
        self.bd = qg.layout("e2m1", n, k, ld=lk, num=e, stride=bs)
        self.vd = qg.layout("e8m0", n, nb, ld=ls, num=e, stride=vs)
        self.batched, self.share = batched, share

    def run(self, g, ws, op=None, alpha=1.0, beta=0.0):
        if ws is not None:
            ws.partials.fill_(float("nan"))
        g.run(op or qg.operation(quant_a=MX, quant_b=MX), alpha, self.a, self.ad, self.sa, self.ud, self.b, self.bd,
              self.sb, self.vd, beta, self.c, self.cd, self.d, self.dd, ws.desc if ws is not None else None)
        return self.result()

    def result(self):
        d = self.d.double().cpu().numpy()
        pad = d[:, self.n:]
        assert (pad == -7).all() if self.out == "i8" else np.isnan(pad).all(), "write past column N"
        return d[:, :self.n]

    def reference(self):
        """(A B^T, |A| |B|^T) in 64 bits; rows that no expert owns are NaN."""
        n = self.n
        if self.counts is None and not self.batched:
            return self.av @ self.bv.T, np.abs(self.av) @ np.abs(self.bv).T
        off = np.concatenate([[0], np.cumsum(self.counts if self.counts is not None else [self.m] * self.batched)])
        ref, ab = np.full((2, len(self.av), n), np.nan)
        for e in range(len(off) - 1):
            a, b = self.av[off[e]:off[e + 1]], self.bv if self.share else self.bv[e * n:(e + 1) * n]
            ref[off[e]:off[e + 1]], ab[off[e]:off[e + 1]] = a @ b.T, np.abs(a) @ np.abs(b).T
        return ref, ab


HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def check(p, d, alpha=1.0, beta=0.0):
    ref, ab = p.reference()
    x = alpha * ref + (beta * p.cv if beta else 0.0)
    if p.out == "f16":
        x, d = np.clip(x, -65504, 65504), np.clip(d, -65504, 65504)
    tol = abs(alpha) * ab * 2.0 ** -24 * (p.k + 2) + 2.0 ** -23 * (abs(alpha) * ab + np.abs(beta * p.cv if beta else 0.0))
    tol = tol + HALF[p.out] * (np.abs(x) + tol) + (2.0 ** -25 if p.out == "f16" else 0.0)
    live = ~np.isnan(ref)
    assert np.isnan(d[~live]).all(), "a row that no expert owns was written"
    bad = ~(np.abs(d - x) <= tol) & live
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), d[bad][:4], x[bad][:4])


KERNELS = [n for n in qg.kernel_names() if n.startswith("mx")]


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 32), (3, 5, 31), (16, 17, 33), (17, 100, 129), (64, 128, 256), (65, 130, 545),
                                   (100, 260, 1000), (128, 256, 4096), (300, 513, 2075), (1, 4096, 14336), (16, 1000, 7168),
                                   (33, 520, 8192), (513, 700, 640)])
def test_product(g, ws, m, n, k):
    p = Problem(m, n, k, seed=m + n + k)
    check(p, p.run(g, ws))


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [7, 90])
def test_output_and_c_types(g, ws, out, c, m):
    p = Problem(m, 72, 384, out=out, seed=9, c=c, extra=1)
    check(p, p.run(g, ws, alpha=0.75, beta=-1.5), 0.75, -1.5)
    check(p, p.run(g, ws, alpha=-1.0), -1.0)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("schedule,split,programs", [(qg.SCHED_DP, 0, 0), (qg.SCHED_SPLITK, 3, 0), (qg.SCHED_STREAMK, 0, 5)])
def test_every_kernel_and_schedule(g, ws, kernel, schedule, split, programs):
    i = qg.kernel_names().index(kernel)
    for m, n, k in ((16, 300, 2944), (13, 129, 2077), (5, 40, 100)):
        p = Problem(m, n, k, out="f32", seed=k, c="bf16")
        op = qg.operation(policy=qg.POLICY_FORCE, schedule=schedule, split_k=split, programs=programs, kernel=i, quant_a=MX,
                          quant_b=MX)
        first = p.run(g, ws, op, alpha=2.0, beta=0.5)
        check(p, first, 2.0, 0.5)
        assert np.array_equal(first, p.run(g, ws, op, alpha=2.0, beta=0.5)), "two runs differ"
        assert int(ws.barriers.abs().sum().item()) == 0


@pytest.mark.parametrize("kernel", [n for n in KERNELS if "skinny" not in n])
@pytest.mark.parametrize("schedule,split", [(qg.SCHED_DP, 0), (qg.SCHED_SPLITK, 2)])
def test_tile_kernels_on_several_tiles(g, ws, kernel, schedule, split):
    i = qg.kernel_names().index(kernel)
    for m, n, k in ((515, 700, 1500), (300, 513, 1024)):
        p = Problem(m, n, k, seed=m)
        op = qg.operation(policy=qg.POLICY_FORCE, schedule=schedule, split_k=split, kernel=i, quant_a=MX, quant_b=MX)
        check(p, p.run(g, ws, op))


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_kernel_grouped(g, ws, kernel):
    i = qg.kernel_names().index(kernel)
    for counts, n, k in (([0, 3, 0, 40, 1, 17, 0], 130, 400), ([5] * 9, 70, 97)):
        p = Problem(sum(counts) + 2, n, k, seed=n, counts=counts)
        check(p, p.run(g, ws, qg.operation(policy=qg.POLICY_FORCE, kernel=i, quant_a=MX, quant_b=MX)))


@pytest.mark.parametrize("counts,n,k", [([0], 64, 64), ([1], 1, 1), ([0, 0, 5, 0], 96, 160), ([130, 1, 0, 300, 64, 2], 264, 512),
                                        ([2] * 64, 256, 1024), ([1] * 200, 33, 65), ([700, 0, 3, 1], 520, 2080)])
@pytest.mark.parametrize("share", [False, True])
def test_grouped(g, ws, counts, n, k, share):
    p = Problem(sum(counts) + 3, n, k, seed=n + k, counts=counts, share=share, extra=1)
    check(p, p.run(g, ws))


def test_grouped_without_rows(g, ws):
    p = Problem(4, 64, 64, counts=[0, 0, 0])
    check(p, p.run(g, ws))


@pytest.mark.parametrize("m", [4, 70, 260])
@pytest.mark.parametrize("share", [False, True])
def test_batched(g, ws, m, share):
    p = Problem(m, 136, 352, seed=m, batched=3, share=share)
    check(p, p.run(g, ws))


@pytest.mark.parametrize("m,counts", [(8, None), (200, None), (90, [30, 0, 60])])
def test_scales_over_their_whole_range(g, ws, m, counts):
    """Scales from 2^-127 to 2^127 that meet to products in range, against sums of a single block."""
    p = Problem(m, 40, 32, out="f32", seed=3, counts=counts)
    r = np.random.default_rng(4)
    e = r.integers(0, 255, (m, 1)).astype(np.uint8)
    p.sa[:, :1] = torch.from_numpy(e).cuda()
    p.av = mx_ref.values(mx_ref.unpack(p.a.cpu().numpy()), e)
    sb = np.full((p.b.shape[0], 1), 127, dtype=np.uint8)
    p.sb[:, :1] = torch.from_numpy(sb).cuda()
    p.bv = mx_ref.values(mx_ref.unpack(p.b.cpu().numpy()), sb)
    with np.errstate(over="ignore"):
        ref, ab = p.reference()
        d = p.run(g, ws)
        live = ~np.isnan(ref)
        tol = 2.0 ** -24 * 36 * ab + 2.0 ** -149 * 36
        big = ab * (1 + 2.0 ** -18) > 3.4028e38  # may overflow on the way
        bad = ~(np.abs(d - ref) <= tol) & live & ~big
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), d[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("m", [5, 150])
def test_nan_scales(g, ws, m):
    """255 is NaN: the outputs of its row (A) or column (B) are NaN, and no others."""
    p = Problem(m, 70, 200, out="f32", seed=8)
    p.sa[2, 3] = 255
    p.sb[11, 6] = 255
    d = p.run(g, ws)
    nan = np.zeros(d.shape, dtype=bool)
    nan[2], nan[:, 11] = True, True
    assert np.array_equal(np.isnan(d), nan)


def test_epilogue(g, ws):
    p = Problem(48, 96, 256, out="f32", seed=5)
    bias = torch.randn(96, device="cuda")
    op = qg.operation(epilogue=qg.EPI_BIAS | qg.EPI_RELU, bias=bias, quant_a=MX, quant_b=MX)
    d = p.run(g, ws, op)
    ref, ab = p.reference()
    want = np.maximum(ref + bias.double().cpu().numpy(), 0)
    assert (np.abs(d - want) <= 2.0 ** -24 * (ab * 260 + 3 * np.abs(want) + 8)).all()


def test_int8_output_codes(g, ws):
    p = Problem(20, 48, 128, out="i8", seed=6)
    scale = torch.full((20,), 2.0 ** -6, device="cuda")
    op = qg.operation(epilogue=qg.EPI_QUANT_I8, row_scale=scale, quant_a=MX, quant_b=MX)
    d = p.run(g, ws, op)
    ref, _ = p.reference()
    pre = ref * 2.0 ** -6
    sure = np.abs(pre - np.floor(pre) - 0.5) > 1e-3
    want = np.clip(np.rint(pre), -128, 127)
    assert np.array_equal(d[sure], want[sure]) and (np.abs(d - want) <= 1).all()


def test_noalloc_matches(g, ws):
    p = Problem(8, 512, 4096, seed=12)
    d = p.run(g, ws).copy()
    p.d.fill_(float("nan"))
    assert g.run_noalloc_raw(qg.operation(quant_a=MX, quant_b=MX), 1.0, p.a, p.ad, p.sa, p.ud, p.b, p.bd, p.sb, p.vd, 0.0,
                             None, None, p.d, p.dd) == qg.OK
    check(p, p.result())
    assert d.shape == p.result().shape


def test_measure_policy(ws):
    g = qg.Gemm()
    p = Problem(24, 256, 1024, seed=13)
    check(p, p.run(g, ws, qg.operation(policy=qg.POLICY_MEASURE, quant_a=MX, quant_b=MX)))
    assert g.cache_size() == 1
    h = qg.Gemm()
    assert h.import_(g.export()) == qg.OK
    check(p, p.run(h, ws, qg.operation(policy=qg.POLICY_REUSE, quant_a=MX, quant_b=MX)))


@pytest.mark.parametrize("m,counts", [(16, None), (300, None), (60, [20, 0, 40])])
def test_graph_replays(g, ws, m, counts):
    p = Problem(m, 256, 2048, seed=14, counts=counts)
    p.run(g, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.run(qg.operation(quant_a=MX, quant_b=MX), 1.0, p.a, p.ad, p.sa, p.ud, p.b, p.bd, p.sb, p.vd, 0.0, None, None, p.d,
              p.dd, ws.desc)
    for i in range(3):
        other = Problem(m, 256, 2048, seed=20 + i, counts=counts)
        p.a.copy_(other.a)
        p.sa.copy_(other.sa)
        p.av = other.av
        p.d.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(p, p.result())


def test_long_rows_past_32_bit_offsets(g, ws):
    """Experts whose weights lie more than 2^32 bytes apart."""
    n, k, e = 64, 256, 3
    stride = (1 << 33) + 2 * n * k  # codes: 2^32 bytes and more
    buf = torch.empty(2 * (stride // 2) + n * k // 2, dtype=torch.uint8, device="cuda")
    p = Problem(30, n, k, seed=15, counts=[10, 10, 10])
    for i in range(e):
        buf[i * (stride // 2):i * (stride // 2) + n * k // 2] = p.b[i * n:(i + 1) * n].reshape(-1)
    p.b, p.bd = buf, qg.layout("e2m1", n, k, num=e, stride=stride)
    check(p, p.run(g, ws))


@pytest.mark.parametrize("n", [1 << 28, (1 << 28) + 64])
def test_columns_past_2_to_the_32_threads(g, ws, n):
    """A row against 2^28 columns and more, each of 32 times 1, some of 32 times -2."""
    q = torch.full((1, 16), 0x22, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 16), 127, dtype=torch.uint8, device="cuda")
    bq = torch.full((n, 16), 0x22, dtype=torch.uint8, device="cuda")
    bq[5::1001] = 0xCC
    bs = torch.full((n, 16), 127, dtype=torch.uint8, device="cuda")
    d = torch.full((1, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    g.run(qg.operation(quant_a=MX, quant_b=MX), 1.0, q, qg.layout("e2m1", 1, 32), s, qg.layout("e8m0", 1, 1), bq,
          qg.layout("e2m1", n, 32), bs, qg.layout("e8m0", n, 1), 0.0, None, None, d, qg.layout("bf16", 1, n), ws.desc)
    want = torch.full((1, n), 32.0, dtype=torch.bfloat16, device="cuda")
    want[0, 5::1001] = -64.0
    assert torch.equal(d, want)
