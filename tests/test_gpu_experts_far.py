"""Operands of the expert block's operators that pass 2^31 elements or 2^32 bytes: what lies far is found, and nothing near it instead."""
import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu
W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def test_combine_from_far_rows(g):
    n, h = 400_000, 8192  # 6.5 GB of results
    r = torch.zeros(n, h, device="cuda", dtype=torch.bfloat16)
    far = [n - 1, 262_143, 262_144, 1, 0, 300_000]
    for i, p in enumerate(far):
        r[p] = float(i + 1)
    back = torch.tensor(far, dtype=torch.int32, device="cuda").view(3, 2)
    w = torch.tensor([[1.0, 0.5], [0.25, 2.0], [4.0, 1.0]], device="cuda")
    y = torch.empty(3, h, device="cuda")
    g.combine(r, qg.layout("bf16", n, h), back, w, qg.layout("f32", 3, 2), y, qg.layout("f32", 3, h))
    assert torch.equal(y, torch.tensor([[1 + 1.0], [0.75 + 8], [20 + 6.0]], device="cuda").expand(3, h))


@pytest.mark.parametrize("act", [qg.MX_IDENTITY, qg.MX_SWIGLU])
def test_quantise_from_far_rows(g, act):
    t, cols = 600_000, 4096  # 4.9 GB of bfloat16
    x = torch.zeros(t, cols, device="cuda", dtype=torch.bfloat16)
    far = [t - 1, 524_288, 524_287, 0, 262_144, t]
    rows = torch.randn(6, cols).bfloat16()
    for i, p in enumerate(far[:5]):
        x[p] = rows[i].cuda()
    rows[5] = 0
    k = cols // (1 + act)
    q, s = torch.empty(6, k, device="cuda", dtype=torch.int8), torch.empty(6, device="cuda")
    idx = torch.tensor(far, dtype=torch.int32, device="cuda")
    g.int_quantize(x, qg.layout("bf16", t, cols), q, qg.layout("i8", 6, k), s, qg.layout("f32", 6, 1), act=act, rows=idx)
    y = rows.double().numpy()
    want, ws = ref.quantise(ref.swiglu(y) if act else y)
    assert np.array_equal(q.cpu().numpy(), want) and np.array_equal(s.cpu().numpy(), ws)


def test_quantise_and_back_to_far_rows(g):
    n, k = 600_000, 4096  # 2.5 GB of codes, 4.9 GB of values
    x = torch.zeros(n, k, device="cuda", dtype=torch.bfloat16)
    at = [0, 1, 524_287, 524_288, n - 1]
    rows = torch.randn(5, k).bfloat16()
    for i, p in enumerate(at):
        x[p] = rows[i].cuda()
    q, s = torch.empty(n, k, device="cuda", dtype=torch.int8), torch.empty(n, device="cuda")
    qd, sd, xd = qg.layout("i8", n, k), qg.layout("f32", n, 1), qg.layout("bf16", n, k)
    g.int_quantize(x, xd, q, qd, s, sd)
    want, ws = ref.quantise(rows.double().numpy())
    assert np.array_equal(q[at].cpu().numpy(), want) and np.array_equal(s[at].cpu().numpy(), ws)
    assert int((s != 0).sum()) == 5 and int(q.view(torch.int64).ne(0).any(-1).sum()) == 5
    x.fill_(7)
    g.int_dequantize(q, qd, s, sd, x, xd)
    values = torch.from_numpy(want.astype(np.float32) * ws[:, None])
    assert (x[at].float().cpu() - values).abs().le(2.0 ** -8 * values.abs() + 2.0 ** -23 * values.abs()).all()
    assert int((x != 0).any(-1).sum()) == 5


@pytest.mark.parametrize("rows", [[3, 2, 4], [40, 0, 300], [2, 700, 900]])
def test_experts_far_apart(g, rows):
    """Weights whose experts lie 2^31 + 2^12 codes apart."""
    n, k, e = 300, 400, 3
    stride = (1 << 31) + (1 << 12)
    r = np.random.default_rng(1)
    b = torch.zeros(2 * stride + n * k, device="cuda", dtype=torch.int8)
    v = torch.zeros(2 * (1 << 20) + n, device="cuda")
    B = r.integers(-128, 128, (e, n, k)).astype(np.int8)
    V = r.uniform(0.001, 0.01, (e, n)).astype(np.float32)
    for i in range(e):
        b[i * stride:i * stride + n * k] = torch.from_numpy(B[i]).cuda().flatten()
        v[i << 20:(i << 20) + n] = torch.from_numpy(V[i]).cuda()
    m = sum(rows)
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    A = r.integers(-128, 128, (m, k)).astype(np.int8)
    U = r.uniform(0.001, 0.01, m).astype(np.float32)
    a, u, offt = torch.from_numpy(A).cuda(), torch.from_numpy(U).cuda(), torch.from_numpy(off).cuda()
    d = torch.empty(m, 304, device="cuda")
    kw = dict(num=e, offsets=offt.data_ptr())
    g.run(qg.operation(quant_a=W8A8, quant_b=W8A8), 1.0, a, qg.layout("i8", m, k, **kw), u, qg.layout("f32", m, 1, **kw), b,
          qg.layout("i8", n, k, num=e, stride=stride), v, qg.layout("f32", n, 1, num=e, stride=1 << 20), 0.0, None, None, d,
          qg.layout("f32", m, n, ld=304, **kw), None)
    got = d[:, :n].double().cpu().numpy()
    for i in range(e):
        at = slice(off[i], off[i + 1])
        want = (A[at].astype(np.float64) @ B[i].astype(np.float64).T) * U[at, None].astype(np.float64) * V[i].astype(np.float64)
        assert (np.abs(got[at] - want) <= 4 * 2.0 ** -24 * np.abs(want)).all(), i
