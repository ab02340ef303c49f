"""MXFP4 products on operands whose sums are exact, so that every output is known to the last bit.

Scales are 1/2, 1 or 2, so products are multiples of 2^-4 of at most 12 * 12 and a sum of K of them is a multiple of 2^-4
of at most 144 K: below 2^24 steps for K <= 7281, whatever the order of its parts. An fp32 output then equals the sum and a
16-bit one its only rounding. One element of K that is lost, doubled or taken from elsewhere is seen at any K.

The persistent loops (grouped, batched, stream-K) are given more tiles than workgroups, with a last round that is
neither full nor a multiple of 8: a workgroup's second tile begins while the first one's stores may still be under
way, its rings start again, and tiles are dealt to the XCDs in rounds."""
import random
import re

import pytest
import torch

import quantized_gemm_bf16_amd as qg

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MX = (qg.QUANT_MX, 32, 1, 0)
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
NAMES = qg.kernel_names()
KERNELS = [n for n in NAMES if n.startswith("mx")]


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


@pytest.fixture(scope="module")
def ws():
    return qg.workspace()


def up(n, to):
    return -(-n // to) * to


def force(kernel, schedule=qg.SCHED_AUTO, **kw):
    return qg.operation(policy=qg.POLICY_FORCE, schedule=schedule, kernel=NAMES.index(kernel), quant_a=MX, quant_b=MX, **kw)


class Operand:
    """Random codes, also past K, and scales, NaN past the last block."""

    def __init__(self, rows, k, gen):
        nb = -(-k // 32)
        self.k, self.nb = k, nb
        self.q = torch.randint(0, 256, (rows, nb * 16), dtype=torch.uint8, device="cuda", generator=gen)
        self.s = torch.full((rows, up(nb, 16)), 255, dtype=torch.uint8, device="cuda")
        self.s[:, :nb] = torch.randint(126, 129, (rows, nb), dtype=torch.uint8, device="cuda", generator=gen)

    def values(self, lo, hi):
        code = torch.stack([self.q[lo:hi] & 15, self.q[lo:hi] >> 4], -1).view(hi - lo, -1).long()
        v = torch.tensor(VALUES + [-x for x in VALUES], dtype=torch.float64, device="cuda")[code]
        return (v * torch.exp2(self.s[lo:hi, :self.nb].double() - 127).repeat_interleave(32, 1))[:, :self.k]


class Product:
    """runs: rows of A of each expert; batched: as many batches of m rows; neither: one product."""

    def __init__(self, m, n, k, out, runs=None, batched=0, seed=0):
        assert k <= 7281
        gen = torch.Generator("cuda").manual_seed(seed)
        e = len(runs) if runs is not None else batched
        self.m, self.n, self.e, self.runs, self.batched = m, n, e, runs, batched
        rows = m * max(1, batched)
        self.a, self.b = Operand(rows, k, gen), Operand(n * max(1, e), k, gen)
        self.d = torch.full((rows, up(n, 8) + 8), float("nan"), dtype=TORCH[out], device="cuda")
        off, lk, ls = 0, up(k, 32), up(self.a.nb, 16)
        if runs is not None:
            self.off = torch.tensor([0] + torch.tensor(runs).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
            off = self.off.data_ptr()

        def rowwise(t, cols, ld):
            return qg.layout(t, m, cols, ld=ld, num=e, offsets=off, stride=m * ld if batched else 0)

        self.layouts = (rowwise("e2m1", k, lk), rowwise("e8m0", self.a.nb, ls), qg.layout("e2m1", n, k, num=e, stride=n * lk if e else 0),
                        qg.layout("e8m0", n, self.a.nb, num=e, stride=n * ls if e else 0), rowwise(out, n, self.d.stride(0)))

    def plan(self, g, op, ws):
        a, u, b, v, d = self.layouts
        return g.plan(op, a, u, b, v, None, d, 1.0, 0.0, ws.desc)

    def run(self, g, op, ws):
        a, u, b, v, d = self.layouts
        g.run(op, 1.0, self.a.q, a, self.a.s, u, self.b.q, b, self.b.s, v, 0.0, None, None, self.d, d, ws.desc)

    def check(self):
        """Every element of D, what lies past column N, and the rows that no expert owns."""
        assert self.d[:, self.n:].isnan().all(), "write past column N"
        at = 0
        for e, rows in enumerate(self.runs if self.runs is not None else [self.m] * max(1, self.batched)):
            b = self.b.values(e * self.n, (e + 1) * self.n).t().contiguous()
            for lo in range(at, at + rows, 4096):
                hi = min(lo + 4096, at + rows)
                want = torch.mm(self.a.values(lo, hi), b).to(self.d.dtype)
                got = self.d[lo:hi, :self.n]
                assert torch.equal(got, want), (e, (got != want).nonzero()[:4].tolist())
            at += rows
        assert self.d[at:].isnan().all(), "a row that no expert owns was written"


def shape(plan):
    return {f: int(re.search(rf"\b{f}=(\d+)", plan)[1]) for f in ("bm", "bn", "bk", "grid")}


def shape_of(kernel, g, ws, **kw):
    return shape(Product(1, 1, 32, "f32", **kw).plan(g, force(kernel), ws))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("schedule,split", [(qg.SCHED_DP, 0), (qg.SCHED_SPLITK, 3), (qg.SCHED_STREAMK, 0)])
@pytest.mark.parametrize("k", [1025, 4096, 7265])
def test_long_sums_exactly(g, ws, kernel, schedule, split, k):
    s = shape_of(kernel, g, ws)
    m = s["bm"] - 3 if "skinny" in kernel else s["bm"] + 5
    p = Product(m, 2 * s["bn"] + 9, k, "f32", seed=k)
    p.run(g, force(kernel, schedule, split_k=split, programs=5 if schedule == qg.SCHED_STREAMK else 0), ws)
    p.check()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("how", ["plain", "grouped", "batched"])
def test_no_columns_to_sum_over(g, ws, kernel, how):
    """K of zero: D is beta C, and zero without C."""
    p = Product(11, 40, 0, "f32", runs=[3, 0, 8] if how == "grouped" else None, batched=2 if how == "batched" else 0)
    p.run(g, force(kernel), ws)
    assert (p.d[:, :40] == 0).all() and p.d[:, 40:].isnan().all()
    c = torch.randn(p.d.shape, device="cuda")
    a, u, b, v, d = p.layouts
    g.run(force(kernel), 1.0, p.a.q, a, p.a.s, u, p.b.q, b, p.b.s, v, 0.5, c, d, p.d, d, ws.desc)
    assert torch.equal(p.d[:, :40], 0.5 * c[:, :40]) and p.d[:, 40:].isnan().all()


def runs_of(tiles, bm, r):
    """Rows of experts that fill `tiles` row tiles between them: ragged, some empty, some of several tiles."""
    runs = []
    while tiles:
        t = min(tiles, r.choice((0, 1, 1, 2, 3, 7)))
        runs.append(t * bm - r.randrange(bm) if t else 0)
        tiles -= t
    return runs + [0]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("out,depth", [("bf16", 0), ("f16", 5), ("f32", 1)])
def test_grouped_over_several_rounds(g, ws, kernel, out, depth):
    r = random.Random(depth)
    s = shape(Product(1, 200000, 32, "f32", runs=[1]).plan(g, force(kernel), ws))  # tiles enough for the largest grid
    columns = 13
    tiles = next(t for t in range(2 * s["grid"] // columns + 1, 1 << 20) if t * columns % s["grid"] % 8)
    runs = runs_of(tiles, s["bm"], r)
    assert sum(-(-x // s["bm"]) for x in runs) == tiles
    p = Product(sum(runs) + 3, columns * s["bn"] - 7, depth * s["bk"] + 37, out, runs=runs, seed=depth)
    assert shape(p.plan(g, force(kernel), ws))["grid"] < tiles * columns // 2
    p.run(g, force(kernel), ws)
    p.check()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("out,depth", [("bf16", 0), ("f16", 5)])
def test_batched_over_several_rounds(g, ws, kernel, out, depth):
    s = shape_of(kernel, g, ws)
    p = Product(2 * s["bm"] - 5, 13 * s["bn"] - 7, depth * s["bk"] + 37, out, batched=81, seed=depth)
    grid, tiles = shape(p.plan(g, force(kernel), ws))["grid"], 81 * 2 * 13
    assert 2 * grid < tiles and tiles % grid % 8
    p.run(g, force(kernel), ws)
    p.check()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_stream_k_programs_of_several_tiles(g, ws, kernel, out):
    s = shape_of(kernel, g, ws)
    m, columns = (s["bm"], 23) if "skinny" in kernel else (3 * s["bm"] - 5, 8)
    p = Product(m, columns * s["bn"] - 7, 3 * s["bk"] + 37, out, seed=3)
    p.run(g, force(kernel, qg.SCHED_STREAMK, programs=5), ws)
    p.check()
    assert int(ws.barriers.abs().sum().item()) == 0


def test_noalloc_split_k(g):
    """A product that the rule cuts along K: the workspace of qg_run_noalloc holds its partial tiles."""
    own = qg.workspace(barriers=qg.noalloc_barriers_size(), partials=qg.noalloc_partials_size())
    op = qg.operation(quant_a=MX, quant_b=MX)
    p = Product(64, 1024, 7200, "f32", seed=7)
    assert "schedule=splitk" in p.plan(g, op, own)
    p.run(g, op, own)
    p.check()
    a, u, b, v, d = p.layouts
    for _ in range(3):
        p.d.fill_(float("nan"))
        assert g.run_noalloc_raw(op, 1.0, p.a.q, a, p.a.s, u, p.b.q, b, p.b.s, v, 0.0, None, None, p.d, d) == qg.OK
        p.check()
