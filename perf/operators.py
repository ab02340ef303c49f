"""What is measured of the MXFP4 operators: four operators of an expert block served in microscaled 4-bit floating point.

  quantise  rows of activations (picked by an index, as a router picks tokens) to E2M1 codes with one E8M0 scale per 32 along K,
            and back to the values they stand for
  gated     silu(gate) * up, quantised in the same pass, and back
  product   D = alpha A B^T + beta C with A and B in MXFP4 and sums in fp32
  grouped   the same product over experts that own ragged runs of A's rows

`run` computes them in plain torch operations; with `own` true it makes the calls of quantized_gemm_bf16_amd instead.

MXFP4: a block of 32 values along K shares the scale 2^(floor(log2 amax) - 2); a value over the scale is rounded to the nearest of
0, 0.5, 1, 1.5, 2, 3, 4, 6 (a tie goes to the even code; past 6 it is 6). Two codes fill a byte, the even k in the low half.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def up(n, to):
    return -(-n // to) * to


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one token's hidden state before a layer: latency alone
        {"name": "quantise 1x4096", "op": "quantise", "tokens": 1, "rows": 1, "k": 4096, "dtype": "bf16"},
        # a ragged batch of odd width, in fp16
        {"name": "quantise 523x7201", "op": "quantise", "tokens": 523, "rows": 523, "k": 7201, "dtype": "f16"},
        # a prompt's tokens, each sent to several experts: rows gathered by the router's index
        {"name": "dispatch 4096to32768x7168", "op": "quantise", "tokens": 4096, "rows": 32768, "k": 7168, "dtype": "bf16"},
        # the gate of a decode batch
        {"name": "gated 16x14336", "op": "gated", "rows": 16, "k": 14336, "dtype": "bf16"},
        # the gate of a prompt
        {"name": "gated 8192x14336", "op": "gated", "rows": 8192, "k": 14336, "dtype": "bf16"},
        # a single token through a down projection
        {"name": "product 1x4096x14336", "op": "product", "m": 1, "n": 4096, "k": 14336, "out": "bf16", "beta": 0.0},
        # a decode batch of 64 through a square projection
        {"name": "product 64x8192x8192", "op": "product", "m": 64, "n": 8192, "k": 8192, "out": "bf16", "beta": 0.0},
        # odd sizes: K ends inside a block, N inside a tile; the result is added to what fp32 C holds
        {"name": "product 333x1001x2075", "op": "product", "m": 333, "n": 1001, "k": 2075, "out": "f32", "beta": 0.5},
        # a prompt through a square projection: bound by the matrix units
        {"name": "product 4096x4096x4096", "op": "product", "m": 4096, "n": 4096, "k": 4096, "out": "bf16", "beta": 0.0},
        # 16 tokens of decode, 8 experts each: every chosen expert's weights are read for a row or two
        {"name": "grouped 64e 128x2048x7168", "op": "grouped", "experts": 64, "rows": 128, "n": 2048, "k": 7168, "out": "bf16", "skew": 0.5},
        # a small mixed batch: ragged experts, some empty, odd widths, fp16
        {"name": "grouped 24e 1501x1000x2080", "op": "grouped", "experts": 24, "rows": 1501, "n": 1000, "k": 2080, "out": "f16", "skew": 1.0},
        # a long prompt over 64 experts
        {"name": "grouped 64e 65536x2048x7168", "op": "grouped", "experts": 64, "rows": 65536, "n": 2048, "k": 7168, "out": "bf16", "skew": 0.5},
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("quantise", "gated", "product", "grouped"))
    k = spread(rng, 64, 14336)
    k = rng.choice((k, up(k, 32), up(k, 128)))
    if op in ("quantise", "gated"):
        rows = spread(rng, 1, max(1, min(65536, 110_000_000 // k)))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        if op == "gated":
            return {"op": op, "rows": rows, "k": k, "dtype": dtype}
        return {"op": op, "tokens": rng.choice((rows, max(1, rows // 8))), "rows": rows, "k": k, "dtype": dtype}
    n = spread(rng, 64, 8192)
    n = rng.choice((n, up(n, 64)))
    out = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "product":
        return {"op": op, "m": spread(rng, 1, 4096), "n": n, "k": k, "out": out, "beta": rng.choice((0.0, 0.0, 0.5))}
    experts = rng.choice((8, 24, 64, 128))
    n = min(n, max(64, 900_000_000 // (experts * k)))
    return {"op": op, "experts": experts, "rows": spread(rng, 1, 16384), "n": n, "k": k, "out": out, "skew": rng.choice((0.0, 0.5, 1.0))}


def counts_of(case):
    """Rows of each expert before the seed deals them out: a few experts are favoured, more so with a larger skew."""
    e = np.arange(case["experts"], dtype=np.float64)
    w = np.exp(-case["skew"] * 4.0 * e / case["experts"])
    edges = np.floor(np.concatenate([[0.0], np.cumsum(w) / w.sum()]) * case["rows"] + 0.5).astype(np.int64)
    return np.diff(edges)


# ---- inputs ------------------------------------------------------------------
def activations(rows, k, dtype, gen):
    """Hidden states: normal, some channels larger, some rows padding (all zero); rows lie at a pitch of 16 bytes."""
    pitch = up(k, 16 // SIZE[dtype])
    x = torch.randn(rows, pitch, device="cuda", generator=gen, dtype=torch.float32)
    x *= torch.exp2(3.0 * torch.rand(pitch, device="cuda", generator=gen) ** 8)
    if rows > 16:
        x[torch.randint(0, rows, (rows // 16,), device="cuda", generator=gen)] = 0
    return x.to(DT[dtype])[:, :k]


def operand(rows, k, std, gen):
    """A matrix in MXFP4 as it is stored: codes (two a byte, rows at a pitch of 16 bytes) and scales (a byte each, the same)."""
    nb = up(k, 32) // 32
    q = torch.zeros(rows, up(k, 32) // 2, device="cuda", dtype=torch.uint8)
    s = torch.zeros(rows, up(nb, 16), device="cuda", dtype=torch.uint8)
    step = max(1, (1 << 27) // max(1, k))
    for r in range(0, rows, step):  # in pieces: the steps between take several times the room of the codes
        n = min(step, rows - r)
        x = torch.zeros(n, nb * 32, device="cuda", dtype=torch.float32)
        x[:, :k] = torch.randn(n, k, device="cuda", generator=gen, dtype=torch.float32) * std
        x = x.view(n, nb, 32)
        e = torch.frexp(x.abs().amax(-1, keepdim=True))[1] - 3
        t = torch.ldexp(x, -e)
        a = t.abs()
        c = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)) | ((t < 0).byte() << 3)
        c = c.view(n, -1, 2)
        q[r:r + n] = c[:, :, 0] | (c[:, :, 1] << 4)
        s[r:r + n, :nb] = (e + 127).clamp(0, 254).squeeze(-1).byte()
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, k = case["op"], case["k"]
    st = {"case": dict(case)}
    if op == "quantise":
        st["x"] = activations(case["tokens"], k, case["dtype"], gen)
        st["index"] = None
        if case["rows"] != case["tokens"]:
            st["index"] = torch.randint(0, case["tokens"], (case["rows"],), device="cuda", generator=gen, dtype=torch.int32)
    elif op == "gated":
        st["x"] = activations(case["rows"], 2 * k, case["dtype"], gen)
    else:
        m, n = (case["m"], case["n"]) if op == "product" else (case["rows"], case["n"])
        st["a"], st["sa"] = operand(m, k, 1.0, gen)
        weights = operand((case["experts"] if op == "grouped" else 1) * n, k, 0.02, gen)
        st["b"], st["sb"] = weights
        pitch = up(n, 8)
        if op == "grouped":
            counts = np.random.RandomState(seed % (1 << 32)).permutation(counts_of(case))
            st["most"] = int(counts.max())
            st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        elif case["beta"]:
            st["c"] = torch.randn(m, pitch, device="cuda", generator=gen)
    if own:
        bind(st)
    return st


# ---- the plain form ------------------------------------------------------------
def rounded(x):
    """The MXFP4 values of x (rows x K, 32 or 64 bits)."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % 32)).view(rows, -1, 32)
    e = torch.frexp(x.abs().amax(-1, keepdim=True))[1] - 3
    t = torch.ldexp(x, -e)
    a = t.abs()
    code = (a > 0.25).long() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    v = torch.tensor(VALUES, device=x.device, dtype=x.dtype)[code]
    return (torch.ldexp(v, e) * torch.sign(x)).view(rows, -1)[:, :k]


def values(q, s, k):
    """The values (32 bits) of stored codes and scales."""
    code = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1, 32).int()
    v = torch.tensor(VALUES + tuple(-x for x in VALUES), device=q.device)[code]
    return torch.ldexp(v, s[:, :v.shape[1], None].int() - 127).view(q.shape[0], -1)[:, :k]


def run(state):
    if own:
        return run_own(state)
    case = state["case"]
    k = case["k"]
    if case["op"] == "quantise":
        x = state["x"] if state["index"] is None else state["x"][state["index"]]
        return rounded(x.float()).to(x.dtype)
    if case["op"] == "gated":
        x = state["x"].double()  # a value next to a rounding border needs more than 32 bits
        g = x[:, :k]
        return rounded(g / (1 + torch.exp(-g)) * x[:, k:]).to(state["x"].dtype)
    a, b = values(state["a"], state["sa"], k), values(state["b"], state["sb"], k)
    if case["op"] == "product":
        d = a @ b.t()
        if case["beta"]:
            d = d + case["beta"] * state["c"][:, :case["n"]]
        return d.to(DT[case["out"]])
    # experts padded to the largest one's rows, as one batched product
    off = state["offsets"].long()
    at = off[:-1, None] + torch.arange(state["most"], device=a.device)
    live = at < off[1:, None]
    d = torch.bmm(a[at.clamp(max=case["rows"] - 1)], b.view(case["experts"], case["n"], k).transpose(1, 2).contiguous())
    return d[live].to(DT[case["out"]])


# ---- the framework's calls -------------------------------------------------------
ENGINE = []  # a program's one handle and workspace


def bind(st):
    """Descriptors and output buffers, as a serving program keeps them next to its weights."""
    import quantized_gemm_bf16_amd as qg

    if not ENGINE:
        ENGINE.extend([qg.Gemm(), qg.workspace()])
    case, k = st["case"], st["case"]["k"]
    nb = up(k, 32) // 32
    if case["op"] in ("quantise", "gated"):
        rows, x = case["rows"], st["x"]
        st["q"] = torch.empty(rows, up(k, 32) // 2, device="cuda", dtype=torch.uint8)
        st["s"] = torch.empty(rows, up(nb, 16), device="cuda", dtype=torch.uint8)
        st["y"] = torch.empty(rows, up(k, 16 // SIZE[case["dtype"]]), device="cuda", dtype=x.dtype)
        st["xd"] = qg.layout(case["dtype"], x.shape[0], x.shape[1], ld=x.stride(0))
        st["qd"], st["sd"] = qg.layout("e2m1", rows, k), qg.layout("e8m0", rows, nb)
        st["yd"] = qg.layout(case["dtype"], rows, k, ld=st["y"].stride(0))
        st["act"] = qg.MX_SWIGLU if case["op"] == "gated" else qg.MX_IDENTITY
        return
    n, grouped = case["n"], case["op"] == "grouped"
    m, experts = (case["rows"], case["experts"]) if grouped else (case["m"], 0)
    off = st["offsets"].data_ptr() if grouped else 0
    st["d"] = torch.empty(m, up(n, 8), device="cuda", dtype=DT[case["out"]])
    st["op"] = qg.operation(quant_a=(qg.QUANT_MX, 32, 1, 0), quant_b=(qg.QUANT_MX, 32, 1, 0))
    st["ad"], st["ud"] = qg.layout("e2m1", m, k, num=experts, offsets=off), qg.layout("e8m0", m, nb, num=experts, offsets=off)
    st["bd"] = qg.layout("e2m1", n, k, num=experts, stride=n * up(k, 32) if grouped else 0)
    st["vd"] = qg.layout("e8m0", n, nb, num=experts, stride=n * up(nb, 16) if grouped else 0)
    st["dd"] = qg.layout(case["out"], m, n, ld=up(n, 8), num=experts, offsets=off)
    st["cd"] = qg.layout("f32", m, n, ld=up(n, 8)) if case.get("beta") else None


def run_own(st):
    case = st["case"]
    engine, space = ENGINE
    if case["op"] in ("quantise", "gated"):
        engine.mx_quantize(st["x"], st["xd"], st["q"], st["qd"], st["s"], st["sd"], act=st["act"], rows=st.get("index"))
        engine.mx_dequantize(st["q"], st["qd"], st["s"], st["sd"], st["y"], st["yd"])
        return st["y"][:, :case["k"]]
    engine.run(st["op"], 1.0, st["a"], st["ad"], st["sa"], st["ud"], st["b"], st["bd"], st["sb"], st["vd"],
               case.get("beta", 0.0), st.get("c"), st["cd"], st["d"], st["dd"], space.desc)
    return st["d"][:, :case["n"]]


# ---- what a pass cannot do without ------------------------------------------------
def work(case):
    k, op = case["k"], case["op"]
    mx = k / 2 + up(k, 32) / 32  # bytes of a row in MXFP4
    if op == "quantise":
        return {"bytes": (min(case["tokens"], case["rows"]) + case["rows"]) * k * SIZE[case["dtype"]], "flops": 0}
    if op == "gated":
        return {"bytes": 3 * case["rows"] * k * SIZE[case["dtype"]], "flops": 0}
    n, size = case["n"], SIZE[case["out"]]
    if op == "product":
        m = case["m"]
        return {"bytes": (m + n) * mx + m * n * (size + (4 if case["beta"] else 0)), "flops": 2 * m * n * k}
    used = int((counts_of(case) > 0).sum())
    return {"bytes": (case["rows"] + used * n) * mx + case["rows"] * n * size, "flops": 2 * case["rows"] * n * k}


# ---- from the definition, in 64 bits ------------------------------------------------
def nearest(x):
    """x in 64 bits to the MXFP4 grid of its blocks, by the spacing of the codes around each value."""
    rows, k = x.shape
    full = torch.zeros(rows, up(k, 32), dtype=torch.float64, device=x.device)
    full[:, :k] = x
    block = full.view(rows, -1, 32)
    top = block.abs().max(-1, keepdim=True).values
    power = (top.view(torch.int64) >> 52) - 1023 - 2  # floor(log2) by the exponent field
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), power.clamp(min=-127).double())
    t = block / scale
    gap = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0)).double()
    return ((torch.round(t / gap) * gap).clamp(-6, 6) * scale).reshape(rows, -1)[:, :k]


def decoded(q, s, k):
    low, high = (q & 15).long(), (q >> 4).long()
    code = torch.empty(q.shape[0], q.shape[1] * 2, dtype=torch.int64, device=q.device)
    code[:, 0::2], code[:, 1::2] = low, high
    exponent, mantissa = (code >> 1) & 3, (code & 1).double()
    v = torch.where(exponent == 0, mantissa * 0.5, (1 + mantissa / 2) * torch.pow(2.0, (exponent - 1).double()))
    v = torch.where(code >= 8, -v, v)[:, :k]
    scale = torch.pow(2.0, s.double() - 127)
    return v * scale.repeat_interleave(32, dim=1)[:, :k]


def exact(case, seed):
    st = prepare(case, seed)
    k = case["k"]
    if case["op"] == "quantise":
        x = st["x"].double()
        return nearest(x if st["index"] is None else x.index_select(0, st["index"].long()))
    if case["op"] == "gated":
        x = st["x"].double()
        return nearest(torch.sigmoid(x[:, :k]) * x[:, :k] * x[:, k:])
    n = case["n"]
    if case["op"] == "product":
        d = torch.mm(decoded(st["a"], st["sa"], k), decoded(st["b"], st["sb"], k).t().contiguous())
        return d + case["beta"] * st["c"][:, :n].double() if case["beta"] else d
    out, off = [], st["offsets"].tolist()
    for e in range(case["experts"]):
        r0, r1 = off[e], off[e + 1]
        a = decoded(st["a"][r0:r1], st["sa"][r0:r1], k)
        out.append(torch.mm(a, decoded(st["b"][e * n:(e + 1) * n], st["sb"][e * n:(e + 1) * n], k).t().contiguous()))
    return torch.cat(out)
