"""MXFP4 entry points on the CPU: refusals of the quantiser, the dequantiser and the product, and the plans. No call
here reaches a launch (fake device addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import quantized_gemm_bf16_amd as qg

FAKE = 1 << 20
I32MAX = (1 << 31) - 1


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


def quant(g, x=FAKE, q=FAKE, s=FAKE, xd="-", qd="-", sd="-", act=0, rows=None, n=4, k=96, dtype="bf16"):
    xd = qg.layout(dtype, n, k * (2 if act == 1 else 1)) if xd == "-" else xd
    qd = qg.layout("e2m1", n, k) if qd == "-" else qd
    sd = qg.layout("e8m0", n, -(-k // 32)) if sd == "-" else sd
    return g.mx_quantize_raw(x, xd, q, qd, s, sd, act=act, rows=rows)


def dequant(g, q=FAKE, s=FAKE, y=FAKE, qd="-", sd="-", yd="-", n=4, k=96, dtype="bf16"):
    qd = qg.layout("e2m1", n, k) if qd == "-" else qd
    sd = qg.layout("e8m0", n, -(-k // 32)) if sd == "-" else sd
    yd = qg.layout(dtype, n, k) if yd == "-" else yd
    return g.mx_dequantize_raw(q, qd, s, sd, y, yd)


def test_layout_default_pitches():
    assert qg.layout("e2m1", 3, 33).ld == 64 and qg.layout("e8m0", 3, 17).ld == 32


def test_null_arguments(g):
    L = qg.lib
    assert L.qg_mx_quantize(None, 0, FAKE, None, None, FAKE, None, FAKE, None, None) == qg.ERR_INVALID_ARG
    assert L.qg_mx_dequantize(None, FAKE, None, FAKE, None, FAKE, None, None) == qg.ERR_INVALID_ARG
    for kw in ({"x": None}, {"q": None}, {"s": None}, {"xd": None}, {"qd": None}, {"sd": None}):
        assert quant(g, **kw) == qg.ERR_INVALID_ARG, kw
    for kw in ({"q": None}, {"s": None}, {"y": None}, {"qd": None}, {"sd": None}, {"yd": None}):
        assert dequant(g, **kw) == qg.ERR_INVALID_ARG, kw
    assert quant(g, act=2) == qg.ERR_INVALID_ARG and quant(g, act=-1) == qg.ERR_INVALID_ARG


@pytest.mark.parametrize("t", ["e4m3", "i8", "i32", "u4", "e2m1", "e8m0"])
def test_value_types(g, t):
    assert quant(g, xd=qg.layout(t, 4, 96, ld=96)) == qg.ERR_UNSUPPORTED
    assert dequant(g, yd=qg.layout(t, 4, 96, ld=96)) == qg.ERR_UNSUPPORTED


def test_operand_types_and_orders(g):
    assert quant(g, qd=qg.layout("u4", 4, 96)) == qg.ERR_UNSUPPORTED
    assert quant(g, sd=qg.layout("f32", 4, 3, ld=16)) == qg.ERR_UNSUPPORTED
    assert quant(g, qd=qg.layout("e2m1", 4, 96, order=qg.COL_MAJOR)) == qg.ERR_UNSUPPORTED
    assert quant(g, xd=qg.layout(9, 4, 96)) == qg.ERR_INVALID_ARG


@pytest.mark.parametrize("act", [0, 1])
def test_shapes(g, act):
    w = 2 if act else 1
    assert quant(g, act=act, xd=qg.layout("bf16", 4, 96 * w + 8)) == qg.ERR_INVALID_ARG
    assert quant(g, act=act, xd=qg.layout("bf16", 5, 96 * w)) == qg.ERR_INVALID_ARG  # without rows: as many as Q
    assert quant(g, act=act, sd=qg.layout("e8m0", 4, 4)) == qg.ERR_INVALID_ARG
    assert quant(g, act=act, sd=qg.layout("e8m0", 3, 3)) == qg.ERR_INVALID_ARG
    assert quant(g, act=act, qd=qg.layout("e2m1", 4, 96, ld=64)) == qg.ERR_INVALID_ARG
    assert quant(g, act=act, xd=qg.layout("bf16", 4, 96 * w, ld=96 * w - 8)) == qg.ERR_INVALID_ARG
    assert quant(g, act=act, qd=qg.layout("e2m1", -1, 96)) == qg.ERR_INVALID_ARG
    assert quant(g, act=act, qd=qg.layout("e2m1", I32MAX + 1, 96)) == qg.ERR_UNSUPPORTED
    assert dequant(g, yd=qg.layout("bf16", 5, 96)) == qg.ERR_INVALID_ARG
    assert dequant(g, yd=qg.layout("bf16", 4, 97, ld=104)) == qg.ERR_INVALID_ARG


def test_alignment(g):
    for kw in ({"x": FAKE + 8}, {"q": FAKE + 4}, {"s": FAKE + 1}, {"rows": FAKE + 2},
               {"xd": qg.layout("bf16", 4, 96, ld=100)}, {"qd": qg.layout("e2m1", 4, 96, ld=112)},
               {"sd": qg.layout("e8m0", 4, 3, ld=8)}):
        assert quant(g, **kw) == qg.ERR_ALIGNMENT, kw
    assert dequant(g, y=FAKE + 8) == qg.ERR_ALIGNMENT
    assert dequant(g, yd=qg.layout("f32", 4, 96, ld=98)) == qg.ERR_ALIGNMENT


def test_batched_layouts_are_refused_and_grouped_ones_count_whole(g):
    assert quant(g, qd=qg.layout("e2m1", 4, 96, num=2, stride=4 * 96)) == qg.ERR_UNSUPPORTED
    st = quant(g, qd=qg.layout("e2m1", 0, 96, num=2, offsets=FAKE), xd=qg.layout("bf16", 7, 96),
               sd=qg.layout("e8m0", 0, 3), rows=FAKE)
    assert st == qg.OK  # no rows: nothing to do


def test_empty_problems_do_nothing(g):
    assert quant(g, x=None, q=None, s=None, n=0) == qg.OK
    assert quant(g, x=None, q=None, s=None, k=0) == qg.OK
    assert dequant(g, q=None, s=None, y=None, n=0) == qg.OK
    assert dequant(g, q=None, s=None, y=None, k=0) == qg.OK


# ---- the product ------------------------------------------------------------------------------
MX = (qg.QUANT_MX, 32, 1, 0)


def operands(m=64, n=128, k=96, num=0, off=0, out="bf16"):
    nb = -(-k // 32)
    bs, vs = (n * -(-k // 32) * 32, n * -(-nb // 16) * 16) if num else (0, 0)
    return {"A": qg.layout("e2m1", m, k, num=num, offsets=off), "U": qg.layout("e8m0", m, nb, num=num, offsets=off),
            "B": qg.layout("e2m1", n, k, num=num, stride=bs), "V": qg.layout("e8m0", n, nb, num=num, stride=vs),
            "D": qg.layout(out, m, n, ld=-(-n // 16) * 16, num=num, offsets=off)}


def run(g, d, op=None, alpha=1.0, beta=0.0, ptr=None, ws=None, C=None, Cd=None):
    p = dict.fromkeys("AUBVD", FAKE)
    p.update(ptr or {})
    return g.run_raw(op or qg.operation(quant_a=MX, quant_b=MX), alpha, p["A"], d["A"], p["U"], d["U"], p["B"], d["B"],
                     p["V"], d["V"], beta, C, Cd, p["D"], d["D"], ws)


def with_(d, **kw):
    d = dict(d)
    d.update(kw)
    return d


def test_product_quant_descriptors(g):
    d = operands()
    for qa, qb in (((0, 0, 0, 0), MX), (MX, (0, 0, 0, 0)), ((qg.QUANT_BLOCK_F32, 32, 1, 0), MX),
                   ((qg.QUANT_MX, 16, 1, 0), MX), (MX, (qg.QUANT_MX, 32, 32, 0)), (MX, (qg.QUANT_MX, 64, 1, 0))):
        assert run(g, d, qg.operation(quant_a=qa, quant_b=qb)) == qg.ERR_UNSUPPORTED


def test_product_types(g):
    d = operands()
    assert run(g, with_(d, B=qg.layout("e4m3", 128, 96))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, A=qg.layout("bf16", 64, 96))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, U=qg.layout("f32", 64, 3, ld=4))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, V=qg.layout("i8", 128, 3, ld=16))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, D=qg.layout("i32", 64, 128))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, D=qg.layout("i8", 64, 128))) == qg.ERR_UNSUPPORTED  # codes only with the epilogue
    assert run(g, d, beta=1.0, C=FAKE, Cd=qg.layout("i32", 64, 128)) == qg.ERR_UNSUPPORTED


def test_product_shapes_and_alignment(g):
    d = operands()
    for kw in ({"U": None}, {"V": None}, {"U": qg.layout("e8m0", 63, 3)}, {"U": qg.layout("e8m0", 64, 4)},
               {"V": qg.layout("e8m0", 127, 3)}, {"V": qg.layout("e8m0", 128, 2)}, {"B": qg.layout("e2m1", 128, 64)},
               {"A": qg.layout("e2m1", 64, 96, ld=64)}, {"D": qg.layout("bf16", 64, 120)}):
        assert run(g, with_(d, **kw)) == qg.ERR_INVALID_ARG, kw
    for name in "AUBVD":
        assert run(g, d, ptr={name: None}) == qg.ERR_INVALID_ARG, name
        assert run(g, d, ptr={name: FAKE + 8}) == qg.ERR_ALIGNMENT, name
    for kw in ({"A": qg.layout("e2m1", 64, 96, ld=97)}, {"B": qg.layout("e2m1", 128, 96, ld=112)},
               {"U": qg.layout("e8m0", 64, 3, ld=20)}, {"V": qg.layout("e8m0", 128, 3, ld=8)}):
        assert run(g, with_(d, **kw)) == qg.ERR_ALIGNMENT, kw
    big = 1 << 25  # 256 rows of codes would pass the kernels' 32-bit offsets
    assert run(g, with_(d, A=qg.layout("e2m1", 64, 96, ld=big))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, V=qg.layout("e8m0", 128, 3, ld=1 << 24))) == qg.ERR_UNSUPPORTED


def test_product_grouped_layouts(g):
    d = operands(num=4, off=FAKE)
    assert run(g, with_(d, V=qg.layout("e8m0", 128, 3, num=2, stride=128 * 16))) == qg.ERR_INVALID_ARG
    assert run(g, with_(d, V=qg.layout("e8m0", 128, 3, num=4, stride=16))) == qg.ERR_INVALID_ARG
    assert run(g, with_(d, U=qg.layout("e8m0", 64, 3, num=4, offsets=2 * FAKE))) == qg.ERR_UNSUPPORTED
    assert run(g, with_(d, B=qg.layout("e2m1", 128, 96, num=4, stride=128 * 96 + 8))) == qg.ERR_ALIGNMENT
    assert run(g, with_(d, V=qg.layout("e8m0", 128, 3, num=4, stride=128 * 16 + 8))) == qg.ERR_ALIGNMENT


def plan(g, d, op=None, ws=None, beta=0.0):
    return g.plan(op or qg.operation(quant_a=MX, quant_b=MX), d["A"], d["U"], d["B"], d["V"], None, d["D"], 1.0, beta, ws)


@pytest.mark.parametrize("m", [1, 16, 17, 64, 100, 300, 4096])
@pytest.mark.parametrize("n,k", [(1, 1), (100, 33), (1001, 2075), (8192, 8192)])
def test_product_plans(g, m, n, k):
    ws = qg.Workspace(FAKE, qg.barriers_size(), FAKE, qg.partials_size())
    for w in (None, ws):
        d = operands(m, n, k)
        assert plan(g, d, ws=w).startswith("kernel=mx")
        d = operands(m, n, k, num=8, off=FAKE)
        assert "schedule=grouped" in plan(g, d, ws=w)


def test_product_every_kernel_and_schedule_plans(g):
    ws = qg.Workspace(FAKE, qg.barriers_size(), FAKE, qg.partials_size())
    d = operands(16, 512, 4096)
    for i, name in enumerate(qg.kernel_names()):
        for s in (qg.SCHED_DP, qg.SCHED_SPLITK, qg.SCHED_STREAMK):
            op = qg.operation(policy=qg.POLICY_FORCE, schedule=s, split_k=2, programs=8, kernel=i, quant_a=MX, quant_b=MX)
            if name.startswith("mx"):
                assert f"kernel={name} " in plan(g, d, op, ws)
            else:
                with pytest.raises(qg.QGemmError) as e:
                    plan(g, d, op, ws)
                assert e.value.status == qg.ERR_NO_KERNEL
    # and no MXFP4 kernel takes another type's operands
    for i, name in enumerate(qg.kernel_names()):
        if name.startswith("mx"):
            op = qg.operation(policy=qg.POLICY_FORCE, kernel=i)
            with pytest.raises(qg.QGemmError):
                g.plan(op, qg.layout("bf16", 16, 4096), None, qg.layout("bf16", 512, 4096), None, None,
                       qg.layout("bf16", 16, 512), 1.0, 0.0, ws)


def test_empty_product(g):
    assert run(g, operands(m=0)) == qg.OK
    assert ctypes.sizeof(qg.Layout) == 56


def test_no_launch_of_2_to_the_32_threads(g):
    """A dispatch counts its threads in 32 bits: 2^28 columns of a row are 2^24 tiles of 256 threads."""
    ws = qg.Workspace(FAKE, qg.barriers_size(), FAKE, qg.partials_size())
    for n in ((1 << 28) - 16, 1 << 28, (1 << 28) + 64):
        p = plan(g, operands(1, n, 32), ws=ws)
        assert "schedule=dp" in p and "_w4_" in p, p  # four waves
        f = dict(x.split("=") for x in p.split())
        assert int(f["tiles"]) == n // 16 and int(f["grid"]) * 256 < 1 << 32, p


def test_rows_tensor(g):
    """What the binding can see of `rows`: entries of another size, apart from each other, or too few are refused."""
    for t in (torch.int64, torch.int16, torch.uint8, torch.float32):
        assert quant(g, rows=torch.zeros(8, dtype=t)) == qg.ERR_UNSUPPORTED, t
    assert quant(g, rows=torch.zeros(4, 2, dtype=torch.int32)[:, 0]) == qg.ERR_INVALID_ARG
    assert quant(g, rows=torch.zeros(3, dtype=torch.int32)) == qg.ERR_INVALID_ARG
    assert quant(g, rows=torch.zeros(0, dtype=torch.int32)) == qg.ERR_INVALID_ARG
    assert quant(g, rows=torch.zeros(4, dtype=torch.int32), qd=None) == qg.ERR_INVALID_ARG
    with pytest.raises(qg.QGemmError) as e:
        g.mx_quantize(FAKE, qg.layout("bf16", 4, 96), FAKE, qg.layout("e2m1", 4, 96), FAKE, qg.layout("e8m0", 4, 3),
                      rows=torch.zeros(4, dtype=torch.int64))
    assert e.value.status == qg.ERR_UNSUPPORTED
    # an int32 tensor passes on: no rows of Q, nothing to do
    assert quant(g, qd=qg.layout("e2m1", 0, 96), sd=qg.layout("e8m0", 0, 3), rows=torch.zeros(1, dtype=torch.int32)) == qg.OK


def test_a_gather_of_no_rows(g):
    """An empty index tensor has no address: with no rows of Q there is nothing to gather, however many rows X has."""
    none = torch.zeros(0, dtype=torch.int32)
    for act in (0, 1):
        assert quant(g, act=act, q=None, s=None, n=0, xd=qg.layout("bf16", 7, 96 * (1 + act)), rows=none) == qg.OK
    assert quant(g, xd=qg.layout("bf16", 7, 96)) == qg.ERR_INVALID_ARG  # with rows of Q they have to agree
