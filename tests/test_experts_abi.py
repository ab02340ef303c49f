"""Entry points around an int8 expert block on the CPU: refusals. No call here reaches a launch (fake device addresses are
never dereferenced)."""
import math

import pytest
import torch

import quantized_gemm_bf16_amd as qg

FAKE = 1 << 20
I32MAX = (1 << 31) - 1
W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)


@pytest.fixture(scope="module")
def g():
    return qg.Gemm()


# ---- int8 quantise / dequantise ---------------------------------------------
def quant(g, x=FAKE, q=FAKE, s=FAKE, xd="-", qd="-", sd="-", act=0, rows=None, n=4, k=96, dtype="bf16"):
    xd = qg.layout(dtype, n, k * (2 if act == 1 else 1)) if xd == "-" else xd
    qd = qg.layout("i8", n, k) if qd == "-" else qd
    sd = qg.layout("f32", n, 1) if sd == "-" else sd
    return g.int_quantize_raw(x, xd, q, qd, s, sd, act=act, rows=rows)


def dequant(g, q=FAKE, s=FAKE, y=FAKE, qd="-", sd="-", yd="-", n=4, k=96, dtype="bf16"):
    qd = qg.layout("i8", n, k) if qd == "-" else qd
    sd = qg.layout("f32", n, 1) if sd == "-" else sd
    yd = qg.layout(dtype, n, k) if yd == "-" else yd
    return g.int_dequantize_raw(q, qd, s, sd, y, yd)


def test_quantise_null_arguments(g):
    L = qg.lib
    assert L.qg_int_quantize(None, 0, FAKE, None, None, FAKE, None, FAKE, None, None) == qg.ERR_INVALID_ARG
    assert L.qg_int_dequantize(None, FAKE, None, FAKE, None, FAKE, None, None) == qg.ERR_INVALID_ARG
    for kw in ({"x": None}, {"q": None}, {"s": None}, {"xd": None}, {"qd": None}, {"sd": None}, {"act": 2}, {"act": -1}):
        assert quant(g, **kw) == qg.ERR_INVALID_ARG, kw
    for kw in ({"q": None}, {"s": None}, {"y": None}, {"qd": None}, {"sd": None}, {"yd": None}):
        assert dequant(g, **kw) == qg.ERR_INVALID_ARG, kw


@pytest.mark.parametrize("t", ["e4m3", "i8", "i32", "u4", "e2m1", "e8m0"])
def test_quantise_types(g, t):
    assert quant(g, xd=qg.layout(t, 4, 96, ld=96)) == qg.ERR_UNSUPPORTED
    assert dequant(g, yd=qg.layout(t, 4, 96, ld=96)) == qg.ERR_UNSUPPORTED
    if t != "i8":
        assert quant(g, qd=qg.layout(t, 4, 96, ld=96)) == qg.ERR_UNSUPPORTED
    assert quant(g, sd=qg.layout(t, 4, 1, ld=16)) == qg.ERR_UNSUPPORTED


def test_quantise_shapes(g):
    bad = qg.ERR_INVALID_ARG
    assert quant(g, xd=qg.layout("bf16", 5, 96)) == bad and quant(g, xd=qg.layout("bf16", 4, 97, ld=104)) == bad
    assert quant(g, act=1, xd=qg.layout("bf16", 4, 96)) == bad
    assert quant(g, sd=qg.layout("f32", 5, 1)) == bad and quant(g, sd=qg.layout("f32", 4, 0, ld=1)) == bad
    assert quant(g, sd=qg.layout("f32", 4, 1, ld=0)) == bad and quant(g, qd=qg.layout("i8", 4, 96, ld=80)) == bad
    assert dequant(g, yd=qg.layout("bf16", 5, 96)) == bad and dequant(g, yd=qg.layout("bf16", 4, 88)) == bad
    assert quant(g, qd=qg.layout("i8", 4, 96, num=2)) == qg.ERR_UNSUPPORTED  # batched
    assert quant(g, xd=qg.layout("bf16", 4, 96, order=qg.COL_MAJOR)) == qg.ERR_UNSUPPORTED
    assert quant(g, k=65552) == qg.ERR_UNSUPPORTED
    assert quant(g, qd=qg.layout("i8", I32MAX + 1, 96)) == qg.ERR_UNSUPPORTED


def test_quantise_alignment(g):
    al = qg.ERR_ALIGNMENT
    assert quant(g, x=FAKE + 8) == al and quant(g, q=FAKE + 8) == al and quant(g, s=FAKE + 2) == al
    assert quant(g, k=100, xd=qg.layout("bf16", 4, 100)) == al and quant(g, qd=qg.layout("i8", 4, 96, ld=100)) == al
    assert quant(g, rows=FAKE + 2) == al
    assert dequant(g, y=FAKE + 8) == al and dequant(g, q=FAKE + 4) == al and dequant(g, s=FAKE + 1) == al


def test_tensors_of_another_type(g):
    un, bad = qg.ERR_UNSUPPORTED, qg.ERR_INVALID_ARG
    assert quant(g, rows=torch.zeros(4, dtype=torch.int64)) == un
    assert quant(g, rows=torch.zeros(3, dtype=torch.int32)) == bad
    assert quant(g, rows=torch.zeros(8, dtype=torch.int32)[::2]) == bad
    assert quant(g, s=torch.zeros(4, dtype=torch.float64)) == un and dequant(g, s=torch.zeros(4, dtype=torch.bfloat16)) == un
    assert route(g, bias=torch.zeros(64, dtype=torch.bfloat16)) == un and route(g, bias=torch.zeros(63)) == bad
    assert route(g, ids=torch.zeros(4, 8, dtype=torch.int64)) == un and route(g, w=torch.zeros(4, 8, dtype=torch.float16)) == un
    i64, i32 = torch.zeros(64, dtype=torch.int64), torch.zeros(31, dtype=torch.int32)
    for at in ("ids", "offsets", "rows", "back"):
        assert group(g, **{at: i64}) == un, at
    assert group(g, rows=i32) == bad and group(g, back=i32) == bad and group(g, offsets=i32, experts=31) == bad
    assert group(g, rows=torch.zeros(64, dtype=torch.int32)[::2]) == bad
    assert combine(g, back=i64) == un and combine(g, back=i32) == bad and combine(g, w=torch.zeros(4, 8, dtype=torch.bfloat16)) == un


# ---- choice --------------------------------------------------------------------
def route(g, r="-", x=FAKE, bias=None, ids=FAKE, w=FAKE, xd="-", idd="-", wd="-", t=4, e=64, k=8, dtype="f32", **kw):
    r = qg.routing(kw.pop("score", 0), k, **kw) if r == "-" else r
    xd = qg.layout(dtype, t, e) if xd == "-" else xd
    idd = qg.layout("i32", t, k) if idd == "-" else idd
    wd = qg.layout("f32", t, k) if wd == "-" else wd
    return g.route_raw(r, x, xd, bias, ids, idd, w, wd)


def test_route_arguments(g):
    bad, un = qg.ERR_INVALID_ARG, qg.ERR_UNSUPPORTED
    assert qg.lib.qg_route(None, None, FAKE, None, None, FAKE, None, FAKE, None, None) == bad
    for kw in ({"r": None}, {"x": None}, {"ids": None}, {"w": None}, {"xd": None}, {"idd": None}, {"wd": None}):
        assert route(g, **kw) == bad, kw
    for kw in ({"score": 2}, {"score": -1}, {"k": 0}, {"k": 65, "e": 64}, {"groups": -1}, {"groups": 5}, {"groups": 8, "top_groups": 0},
               {"groups": 8, "top_groups": 9}, {"groups": 8, "top_groups": 1, "k": 9}, {"groups": 8, "top_groups": 2, "group_best": 3},
               {"groups": 8, "top_groups": 2, "group_best": 0}, {"scale": math.inf}, {"scale": math.nan}, {"e": 0, "k": 1}):
        assert route(g, **kw) == bad, kw
    for kw in ({"k": 33}, {"e": 1028, "dtype": "f32"}, {"e": 130, "groups": 65, "top_groups": 65, "xd": qg.layout("f32", 4, 130, ld=132)},
               {"e": 1020, "groups": 5, "top_groups": 5}, {"xd": qg.layout("i32", 4, 64)}, {"idd": qg.layout("f32", 4, 8)},
               {"wd": qg.layout("bf16", 4, 8)}, {"xd": qg.layout("f32", 4, 64, num=2)}):
        assert route(g, **kw) == un, kw
    for kw in ({"idd": qg.layout("i32", 5, 8)}, {"idd": qg.layout("i32", 4, 7)}, {"wd": qg.layout("f32", 4, 9)}, {"wd": qg.layout("f32", 4, 8, ld=7)},
               {"xd": qg.layout("f32", 4, 64, ld=60)}):
        assert route(g, **kw) == bad, kw
    for kw in ({"x": FAKE + 4}, {"e": 62, "xd": qg.layout("f32", 4, 62)}, {"ids": FAKE + 2}, {"w": FAKE + 1}, {"bias": FAKE + 2}):
        assert route(g, **kw) == qg.ERR_ALIGNMENT, kw
    assert route(g, t=0, x=None, ids=None, w=None) == qg.OK
    if not torch.cuda.is_available():
        assert route(g) == qg.ERR_HIP and route(g, e=1024, groups=64, top_groups=8, group_best=2) == qg.ERR_HIP
        assert route(g, e=16, k=8, groups=0, top_groups=0, group_best=0) == qg.ERR_HIP  # no groups: their fields are not looked at


# ---- sorting ---------------------------------------------------------------------
def group(g, experts=32, ids=FAKE, idd="-", offsets=FAKE, rows=FAKE, back=FAKE, ws=None, t=4, k=8):
    return g.group_rows_raw(experts, ids, qg.layout("i32", t, k) if idd == "-" else idd, offsets, rows, back, ws)


def test_group_arguments(g):
    bad, un = qg.ERR_INVALID_ARG, qg.ERR_UNSUPPORTED
    for kw in ({"experts": 0}, {"experts": -4}, {"ids": None}, {"idd": None}, {"offsets": None}, {"rows": None}, {"back": None},
               {"idd": qg.layout("i32", 4, 8, ld=7)}):
        assert group(g, **kw) == bad, kw
    for kw in ({"experts": 1024}, {"idd": qg.layout("f32", 4, 8)}, {"t": 1 << 28, "k": 5}, {"idd": qg.layout("i32", 4, 8, num=2)}):
        assert group(g, **kw) == un, kw
    for kw in ({"ids": FAKE + 2}, {"offsets": FAKE + 1}, {"rows": FAKE + 2}, {"back": FAKE + 3}):
        assert group(g, **kw) == qg.ERR_ALIGNMENT, kw
    big = dict(t=1025, k=8)
    assert group(g, **big) == qg.ERR_WORKSPACE
    assert group(g, ws=qg.Workspace(FAKE, 1 << 20, FAKE, 100), **big) == qg.ERR_WORKSPACE
    assert group(g, ws=qg.Workspace(FAKE, 1 << 20, FAKE + 4, 1 << 25), **big) == qg.ERR_ALIGNMENT
    if not torch.cuda.is_available():
        assert group(g) == qg.ERR_HIP and group(g, ws=qg.Workspace(None, 0, FAKE, 1024 * 32), **big) == qg.ERR_HIP


# ---- combination -------------------------------------------------------------------
def combine(g, r=FAKE, rd="-", back=FAKE, w=FAKE, wd="-", y=FAKE, yd="-", beta=0.0, c=None, cd=None, t=4, k=8, h=64):
    rd = qg.layout("bf16", t * k, h) if rd == "-" else rd
    wd = qg.layout("f32", t, k) if wd == "-" else wd
    yd = qg.layout("bf16", t, h) if yd == "-" else yd
    return g.combine_raw(r, rd, back, w, wd, y, yd, beta, c, cd)


def test_combine_arguments(g):
    bad, un = qg.ERR_INVALID_ARG, qg.ERR_UNSUPPORTED
    c4 = qg.layout("f32", 4, 64)
    for kw in ({"r": None}, {"rd": None}, {"back": None}, {"w": None}, {"wd": None}, {"y": None}, {"yd": None}, {"beta": 1.0}, {"beta": 1.0, "c": FAKE},
               {"beta": 1.0, "cd": c4}, {"beta": math.nan}, {"beta": math.inf, "c": FAKE, "cd": c4}, {"wd": qg.layout("f32", 5, 8)},
               {"rd": qg.layout("bf16", 32, 72)}, {"beta": 1.0, "c": FAKE, "cd": qg.layout("f32", 5, 64)}, {"yd": qg.layout("bf16", 4, 64, ld=56)}):
        assert combine(g, **kw) == bad, kw
    for kw in ({"rd": qg.layout("i8", 32, 64)}, {"yd": qg.layout("i32", 4, 64)}, {"wd": qg.layout("bf16", 4, 8)}, {"beta": 1.0, "c": FAKE, "cd": qg.layout("i8", 4, 64)},
               {"yd": qg.layout("bf16", 4, 64, num=2)}):
        assert combine(g, **kw) == un, kw
    for kw in ({"r": FAKE + 8}, {"y": FAKE + 8}, {"w": FAKE + 2}, {"back": FAKE + 2}, {"beta": 1.0, "c": FAKE + 4, "cd": c4}, {"h": 60, "rd": qg.layout("bf16", 32, 60)}):
        assert combine(g, **kw) == qg.ERR_ALIGNMENT, kw
    assert combine(g, t=0, r=None, back=None, w=None, y=None) == qg.OK


# ---- grouped and batched int8 products ----------------------------------------------
def product(g, e=4, m=40, n=64, k=96, off=FAKE, ud="-", vd="-", v=FAKE, u=FAKE, out="bf16", **kw):
    ad = qg.layout("i8", m, k, num=e, offsets=off, stride=0 if off else m * k)
    bd = qg.layout("i8", n, k, num=e, stride=n * k)
    dd = qg.layout(out, m, n, num=e, offsets=off, stride=0 if off else m * n)
    ud = qg.layout("f32", m, 1, num=e, offsets=off, stride=0 if off else m) if ud == "-" else ud
    vd = qg.layout("f32", n, 1, num=e, stride=n) if vd == "-" else vd
    return g.run_raw(qg.operation(quant_a=W8A8, quant_b=W8A8), 1.0, FAKE, ad, u, ud, FAKE, bd, v, vd, 0.0, None, None, FAKE, dd, None)


def test_products(g):
    bad, un = qg.ERR_INVALID_ARG, qg.ERR_UNSUPPORTED
    for kw in ({"vd": qg.layout("f32", 64, 1)}, {"vd": qg.layout("f32", 64, 1, num=4, stride=63)}, {"vd": qg.layout("f32", 63, 1, num=4, stride=64)},
               {"ud": qg.layout("f32", 39, 1, num=4, offsets=FAKE)}, {"u": None}, {"v": None}, {"vd": None}, {"ud": None}):
        assert product(g, **kw) == bad, kw
    for kw in ({"ud": qg.layout("f32", 40, 1, num=4, offsets=FAKE + 64)}, {"off": 0, "ud": qg.layout("f32", 40, 1, num=4, stride=41)},
               {"off": 0, "ud": qg.layout("f32", 40, 1, stride=40)}, {"e": 1024}, {"out": "i32"}):
        assert product(g, **kw) == un, kw
    assert product(g, u=FAKE + 2) == qg.ERR_ALIGNMENT and product(g, v=FAKE + 1) == qg.ERR_ALIGNMENT
    ad, bd = qg.layout("i8", 40, 96, num=4, offsets=FAKE), qg.layout("i8", 64, 96, num=4, stride=64 * 96)
    ud, vd = qg.layout("f32", 40, 1, num=4, offsets=FAKE), qg.layout("f32", 64, 1, num=4, stride=64)
    op = qg.operation(quant_a=W8A8, quant_b=W8A8)
    plan = g.plan(op, ad, ud, bd, vd, None, qg.layout("bf16", 40, 64, num=4, offsets=FAKE), 1.0, 0.0)
    assert "_I8_" in plan and "schedule=grouped" in plan
