"""The 256 x 256 int8 tile on operands that pass the memory-side cache (256 MB), where a wave touches the lines of k-tiles ahead of
the ring: ragged ends of rows and columns, K that is no multiple of 16 with extreme codes behind it, several tiles per workgroup.
int32 results are equal to the sums (in float64, which holds them). With scales four roundings of fp32 and half a step of the type."""
import pytest
import torch

import quantized_gemm_bf16_amd as qg

pytestmark = pytest.mark.gpu
BIG = "tile_I8_256x256x128b_w2x4_s2"
W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)
PAST = 256 << 20


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


@pytest.fixture(scope="module")
def ws():
    return qg.workspace()


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def codes(rows, k, pitch, fill, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.full((rows, pitch), fill, device="cuda", dtype=torch.int8)
    x[:, :k] = torch.randint(-128, 128, (rows, k), device="cuda", dtype=torch.int8, generator=gen)
    return x


def check(d, sums, scaled, u, v):
    if not scaled:
        assert torch.equal(d, sums.to(torch.int32))
        return
    x = sums * u.double()[:, None] * v.double()
    tol = 4.01 * 2.0 ** -24 * x.abs()
    assert ((d.double() - x).abs() <= tol + 2.0 ** -8 * (x.abs() + tol)).all()


def operands(m, n, k, e, scaled, seed):
    pitch = -(-k // 16) * 16 + 16
    A, B = codes(m, k, pitch, 127, seed), codes(max(e, 1) * n, k, pitch, -128, seed + 1)
    assert A.numel() + B.numel() > PAST
    u, v = torch.rand(m, device="cuda") * 0.01, torch.rand(max(e, 1) * n, device="cuda") * 0.01
    ldd = -(-n // 16) * 16
    d = torch.full((m, ldd), -77, device="cuda", dtype=torch.bfloat16 if scaled else torch.int32)
    quant = dict(quant_a=W8A8, quant_b=W8A8) if scaled else {}
    return A, B, u, v, d, pitch, dict(policy=qg.POLICY_FORCE, kernel=qg.kernel_names().index(BIG), **quant)


@pytest.mark.parametrize("scaled", [False, True])
def test_experts(g, ws, scaled):
    counts, n, k = [1300, 0, 255, 2100, 1, 1024, 3001, 514], 1990, 20009
    e, m = len(counts), sum(counts) + 3
    A, B, u, v, d, pitch, kw_op = operands(m, n, k, e, scaled, 1)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    kw = dict(num=e, offsets=off.data_ptr())
    args = (qg.operation(**kw_op), 1.0, A, qg.layout("i8", m, k, ld=pitch, **kw), u, qg.layout("f32", m, 1, **kw),
            B, qg.layout("i8", n, k, ld=pitch, num=e, stride=n * pitch), v, qg.layout("f32", n, 1, num=e, stride=n), 0.0, None, None, d, qg.layout("bf16" if scaled else "i32", m, n, ld=d.shape[1], **kw), ws.desc)
    g.run(*args)
    first = d.clone()
    assert (d[:, n:] == -77).all() and (d[-3:] == -77).all(), "write past column N or behind the last expert"
    at = 0
    for i, c in enumerate(counts):
        if c:
            sums = A[at:at + c, :k].double() @ B[i * n:(i + 1) * n, :k].double().t().contiguous()
            check(d[at:at + c, :n], sums, scaled, u[at:at + c], v[i * n:(i + 1) * n])
        at += c
    g.run(*args)
    assert torch.equal(d, first)


@pytest.mark.parametrize("scaled", [False, True])
def test_plain_products(g, ws, scaled):
    m, n, k = 1301, 1490, 100041  # (36 tiles: three parts of each fit into the workspace)
    A, B, u, v, d, pitch, kw_op = operands(m, n, k, 0, scaled, 3)
    sums = A[:, :k].double() @ B[:, :k].double().t().contiguous()
    for schedule, kw in ((qg.SCHED_DP, {}), (qg.SCHED_SPLITK, dict(split_k=3)), (qg.SCHED_STREAMK, dict(programs=50))):
        d.fill_(-77)
        g.run(qg.operation(schedule=schedule, **kw, **kw_op), 1.0, A, qg.layout("i8", m, k, ld=pitch), u, qg.layout("f32", m, 1),
              B, qg.layout("i8", n, k, ld=pitch), v, qg.layout("f32", n, 1), 0.0, None, None, d, qg.layout("bf16" if scaled else "i32", m, n, ld=d.shape[1]), ws.desc)
        assert (d[:, n:] == -77).all(), "write past column N"
        check(d[:, :n], sums, scaled, u, v)
    assert not ws.barriers.any()
