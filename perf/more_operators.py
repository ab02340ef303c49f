"""What is measured of an expert block served in 8-bit integers: the operators before, between and behind its products.

  route     each token's experts and their weights from the router's logits (softmax or sigmoid, bias, groups)
  group     the chosen experts sorted into runs: offsets, source rows, and where each choice went
  quantise  rows of activations (picked by an index), or silu(gate) * up, to int8 with a scale per row, and back to values
  product   D = alpha (A U) (B V)^T + beta C over experts that own ragged runs of A's rows; A, B int8, U per row, V per channel
  combine   each token's rows of the experts' results, weighted and added, plus what a shared expert gave

`run` computes them in plain torch operations; with `own` true it makes the calls of quantized_gemm_bf16_amd instead.

Choice: score p = softmax(logits) or sigmoid(logits), key = p + bias (the logit itself where there is no bias: the same
order). An expert whose logit is -inf or NaN, or whose key is, is never chosen. With groups of E / G experts, a group's
standing is its best key, or the sum of its two best; the best `top_groups` groups keep their experts. The top_k best keys are
chosen, best first, ties to the lowest index; id -1 and weight 0 where too few are left. Weight: p, over the chosen ones' sum
where renormalised, times scale.

Int8: a row's scale is fp32(amax / 127); a code is the value over the scale, rounded half to even.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def up(n, to):
    return -(-n // to) * to


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one token's choice, from a plain softmax: latency alone
        {"name": "route 1x64", "op": "route", "tokens": 1, "experts": 64, "dtype": "f32", "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "group_best": 1, "top_k": 8, "renorm": True, "scale": 1.0},
        # a prompt's choice among many experts in groups, with a bias for balance
        {"name": "route 16384x256 groups", "op": "route", "tokens": 16384, "experts": 256, "dtype": "f32", "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_best": 2, "top_k": 8, "renorm": True, "scale": 2.5},
        # a decode batch sorted by expert
        {"name": "group 16x8 of 64", "op": "group", "tokens": 16, "top_k": 8, "experts": 64, "of": 64},
        # a long prompt sorted by expert
        {"name": "group 65536x8 of 256", "op": "group", "tokens": 65536, "top_k": 8, "experts": 256, "of": 256},
        # one token's hidden state before a layer: latency alone
        {"name": "quantise 1x4096", "op": "quantise", "tokens": 1, "rows": 1, "k": 4096, "dtype": "bf16"},
        # a prompt's tokens, each sent to several experts: rows gathered by the router's index
        {"name": "dispatch 4096to32768x7168", "op": "quantise", "tokens": 4096, "rows": 32768, "k": 7168, "dtype": "bf16"},
        # the gate of a prompt
        {"name": "gated 8192x14336", "op": "gated", "rows": 8192, "k": 14336, "dtype": "bf16"},
        # 16 tokens of decode, 8 experts each: every chosen expert's weights are read for a row or two
        {"name": "product 64e 128x2048x7168", "op": "product", "experts": 64, "rows": 128, "n": 2048, "k": 7168, "out": "bf16", "skew": 0.5, "beta": 0.0},
        # a small mixed batch: ragged experts, some empty, odd widths, added to fp16 results that are there already
        {"name": "product 24e 1501x1000x2075", "op": "product", "experts": 24, "rows": 1501, "n": 1000, "k": 2075, "out": "f16", "skew": 1.0, "beta": 1.0},
        # a long prompt over 64 experts: bound by the matrix units
        {"name": "product 64e 65536x2048x7168", "op": "product", "experts": 64, "rows": 65536, "n": 2048, "k": 7168, "out": "bf16", "skew": 0.5, "beta": 0.0},
        # a decode batch put together again
        {"name": "combine 16x8x7168", "op": "combine", "tokens": 16, "top_k": 8, "k": 7168, "dtype": "bf16", "out": "bf16", "held": 1.0, "shared": False},
        # a prompt put together again, with a shared expert's results
        {"name": "combine 8192x8x7168 shared", "op": "combine", "tokens": 8192, "top_k": 8, "k": 7168, "dtype": "bf16", "out": "bf16", "held": 1.0, "shared": True},
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("route", "group", "quantise", "gated", "product", "combine"))
    top_k = rng.choice((1, 2, 4, 6, 8, 10))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * rng.choice((rng.randint(2, 512 // groups), max(16, 64 // groups), 256 // groups))
        top_groups = rng.randint(1, groups)
        return {"op": op, "tokens": spread(rng, 1, 16384 * 256 // max(experts, 256)), "experts": experts, "dtype": rng.choice(("f32", "f32", "bf16", "f16")),
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "group_best": rng.choice((1, 2)), "top_k": min(top_k, top_groups * (experts // groups)), "renorm": rng.random() < 0.7,
                "scale": rng.choice((1.0, 2.5))}
    if op == "group":
        of = rng.choice((8, 60, 64, 128, 256, rng.randint(11, 512)))
        top_k = min(top_k, of)
        return {"op": op, "tokens": spread(rng, 1, 65536 * 8 // max(top_k, 8)), "top_k": top_k, "experts": max(1, of // rng.choice((1, 1, 4, 8))), "of": of}
    k = spread(rng, 64, 14336)
    k = rng.choice((k, up(k, 32), up(k, 128)))
    if op in ("quantise", "gated"):
        rows = spread(rng, 1, max(1, min(65536, 110_000_000 // k)))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        if op == "gated":
            return {"op": op, "rows": rows, "k": k, "dtype": dtype}
        return {"op": op, "tokens": rng.choice((rows, max(1, rows // 8))), "rows": rows, "k": k, "dtype": dtype}
    if op == "combine":
        return {"op": op, "tokens": spread(rng, 1, max(1, min(65536, 450_000_000 // (k * top_k)))), "top_k": top_k, "k": k, "dtype": rng.choice(("bf16", "f16", "f32")),
                "out": rng.choice(("bf16", "f16", "f32")), "held": rng.choice((1.0, 0.25)), "shared": rng.random() < 0.5}
    n = spread(rng, 64, 8192)
    n = rng.choice((n, up(n, 64)))
    experts = rng.choice((8, 24, 64, 128))
    n = min(n, max(64, 900_000_000 // (experts * k)))
    return {"op": op, "experts": experts, "rows": spread(rng, 1, 16384), "n": n, "k": k, "out": rng.choice(("bf16", "bf16", "f16", "f32")),
            "skew": rng.choice((0.0, 0.5, 1.0)), "beta": rng.choice((0.0, 0.0, 1.0))}


def counts_of(case):
    """Rows of each expert before the seed deals them out: a few experts are favoured, more so with a larger skew."""
    e = np.arange(case["experts"], dtype=np.float64)
    w = np.exp(-case["skew"] * 4.0 * e / case["experts"])
    edges = np.floor(np.concatenate([[0.0], np.cumsum(w) / w.sum()]) * case["rows"] + 0.5).astype(np.int64)
    return np.diff(edges)


# ---- inputs ------------------------------------------------------------------
def pitched(rows, cols, dtype, gen):
    """Normal values; rows lie at a pitch of 16 bytes."""
    return torch.randn(rows, up(cols, 16 // SIZE[dtype]), device="cuda", generator=gen, dtype=torch.float32).to(DT[dtype])[:, :cols]


def activations(rows, k, dtype, gen):
    """Hidden states: normal, some channels larger, some rows padding (all zero); rows lie at a pitch of 16 bytes."""
    pitch = up(k, 16 // SIZE[dtype])
    x = torch.randn(rows, pitch, device="cuda", generator=gen, dtype=torch.float32)
    x *= torch.exp2(3.0 * torch.rand(pitch, device="cuda", generator=gen) ** 8)
    if rows > 16:
        x[torch.randint(0, rows, (rows // 16,), device="cuda", generator=gen)] = 0
    return x.to(DT[dtype])[:, :k]


def operand(rows, k, gen):
    """An int8 matrix as it is stored, rows at a pitch of 16 bytes: normal values whose largest is about 4 deviations out."""
    q = torch.empty(rows, up(k, 16), device="cuda", dtype=torch.int8)
    step = max(1, (1 << 27) // q.shape[1])
    for r in range(0, rows, step):  # in pieces: the steps between take several times the room of the codes
        x = torch.randn(min(step, rows - r), q.shape[1], device="cuda", generator=gen)
        q[r:r + step] = (x * 32).round_().clamp_(-127, 127).to(torch.int8)
    return q


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "route":
        t, e = case["tokens"], case["experts"]
        x = 1.5 * torch.randn(t, e, device="cuda", generator=gen) + 0.5 * torch.randn(e, device="cuda", generator=gen)
        if t > 16:  # padding of a batch: nothing may be chosen
            x[torch.randint(0, t, (t // 16,), device="cuda", generator=gen)] = -math.inf
        st["logits"] = torch.zeros(t, up(e, 16 // SIZE[case["dtype"]]), device="cuda", dtype=DT[case["dtype"]])[:, :e]
        st["logits"].copy_(x)
        st["bias"] = 0.1 * torch.randn(e, device="cuda", generator=gen) if case["bias"] else None
    elif op == "group":
        taste = torch.randn(case["tokens"], case["of"], device="cuda", generator=gen) + torch.randn(case["of"], device="cuda", generator=gen)
        ids = taste.topk(case["top_k"], -1).indices - (case["of"] - case["experts"]) // 2  # the experts held here are some in the middle
        st["ids"] = ids.to(torch.int32)
    elif op == "quantise":
        st["x"] = activations(case["tokens"], case["k"], case["dtype"], gen)
        st["index"] = None
        if case["rows"] != case["tokens"]:
            st["index"] = torch.randint(0, case["tokens"], (case["rows"],), device="cuda", generator=gen, dtype=torch.int32)
    elif op == "gated":
        st["x"] = activations(case["rows"], 2 * case["k"], case["dtype"], gen)
    elif op == "product":
        m, n, k = case["rows"], case["n"], case["k"]
        st["a"], st["b"] = operand(m, k, gen), operand(case["experts"] * n, k, gen)
        st["u"] = (0.5 + torch.rand(m, device="cuda", generator=gen)) / 32
        st["v"] = (0.5 + torch.rand(case["experts"] * n, device="cuda", generator=gen)) * (0.02 / 32)
        st["c"] = pitched(m, n, case["out"], gen) if case["beta"] else None
        counts = np.random.RandomState(seed % (1 << 32)).permutation(counts_of(case))
        st["most"] = int(counts.max())
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    else:
        n = case["tokens"] * case["top_k"]
        st["r"] = pitched(n, case["k"], case["dtype"], gen)
        gone = torch.rand(n, device="cuda", generator=gen) >= case["held"]  # choices of experts that another process holds
        back = torch.randperm(n, device="cuda", generator=gen).to(torch.int32)
        st["back"] = torch.where(gone, -1, back).view(case["tokens"], case["top_k"])
        st["w"] = torch.rand(case["tokens"], case["top_k"], device="cuda", generator=gen) + 0.1
        st["w"] /= st["w"].sum(-1, keepdim=True)
        st["c"] = pitched(case["tokens"], case["k"], case["out"], gen) if case["shared"] else None
    if own:
        bind(st)
    return st


# ---- the plain form ------------------------------------------------------------
def best(key, n):
    """Places of the n largest along the last axis, largest first, ties to the lowest."""
    return key.sort(dim=-1, descending=True, stable=True).indices[..., :n]


def route(state):
    case = state["case"]
    x = state["logits"].double()  # a key next to another one needs more than 32 bits
    dead = torch.isnan(x) | (x == -math.inf)
    if case["score"] == "softmax":
        p = torch.exp(x - x.masked_fill(dead, -math.inf).amax(-1, keepdim=True)).masked_fill(dead, 0.0)
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        p = (1 / (1 + torch.exp(-x))).masked_fill(dead, 0.0)
    standing = p if state["bias"] is None else p + state["bias"].double()
    key = x if state["bias"] is None else standing
    key = key.masked_fill(dead, -math.inf)
    if case["groups"] > 1:
        split = (case["tokens"], case["groups"], -1)
        if case["group_best"] == 1:
            group = key.view(split).amax(-1)
        else:
            two = standing.masked_fill(dead, -math.inf).view(split).sort(-1, descending=True).values[..., :2]
            group = two.masked_fill(two == -math.inf, 0.0).sum(-1).masked_fill(two[..., 0] == -math.inf, -math.inf)
        kept = torch.zeros(split[:2], device=x.device, dtype=torch.bool).scatter_(1, best(group, case["top_groups"]), True)
        key = key.view(split).masked_fill(~kept[..., None], -math.inf).view(case["tokens"], -1)
    ids = best(key, case["top_k"])
    live = key.gather(1, ids) > -math.inf
    w = p.gather(1, ids) * live
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return torch.where(live, ids, -1).to(torch.int32), (w * case["scale"]).float()


def group(state):
    case, flat = state["case"], state["ids"].flatten().long()
    live = (flat >= 0) & (flat < case["experts"])
    key, order = torch.where(live, flat, case["experts"]).sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(case["experts"] + 1, device=key.device))
    rows = torch.where(key < case["experts"], order // case["top_k"], -1)
    back = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    return offsets.int(), rows.int(), torch.where(live, back, -1).int().view(case["tokens"], case["top_k"])


def rounded(x):
    """The values of x's rows (64 bits) in int8."""
    s = (x.abs().amax(-1, keepdim=True) / 127).float().double()
    q = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)), 0.0)
    return q.clamp(-127, 127) * s


def run(state):
    if own:
        return run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "route":
        return route(state)
    if op == "group":
        return group(state)
    if op == "quantise":
        x = state["x"] if state["index"] is None else state["x"][state["index"]]
        return rounded(x.double()).to(x.dtype)  # a value next to a rounding border needs more than 32 bits
    if op == "gated":
        x, k = state["x"].double(), case["k"]
        g = x[:, :k]
        return rounded(g / (1 + torch.exp(-g)) * x[:, k:]).to(state["x"].dtype)
    if op == "combine":
        r = state["r"][state["back"].clamp(min=0)].float()
        y = (r * (state["w"] * (state["back"] >= 0))[..., None]).sum(1)
        return (y if state["c"] is None else y + state["c"].float()).to(DT[case["out"]])
    # experts padded to the largest one's rows, as one batched product
    k, off = case["k"], state["offsets"].long()
    at = off[:-1, None] + torch.arange(state["most"], device=off.device)
    live = at < off[1:, None]
    a = state["a"][at.clamp(max=case["rows"] - 1), :k].float()
    b = state["b"].view(case["experts"], case["n"], -1)[:, :, :k].float().transpose(1, 2).contiguous()
    d = torch.bmm(a, b).mul_(state["v"].view(case["experts"], 1, -1))[live] * state["u"][:, None]
    return (d if state["c"] is None else d + case["beta"] * state["c"].float()).to(DT[case["out"]])


# ---- the framework's calls -------------------------------------------------------
ENGINE = []  # a program's one handle and workspace


def bind(st):
    """Descriptors and output buffers, as a serving program keeps them next to its weights."""
    import quantized_gemm_bf16_amd as qg

    if not ENGINE:
        ENGINE.extend([qg.Gemm(), qg.workspace()])
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        t, top_k = case["tokens"], case["top_k"]
        st["routing"] = qg.routing(qg.ROUTE_SOFTMAX if case["score"] == "softmax" else qg.ROUTE_SIGMOID, top_k, groups=case["groups"],
                                   top_groups=case["top_groups"], group_best=case["group_best"], renormalize=case["renorm"], scale=case["scale"])
        st["ids"] = torch.empty(t, top_k, device="cuda", dtype=torch.int32)
        st["w"] = torch.empty(t, top_k, device="cuda")
        st["ld"] = qg.layout(case["dtype"], t, case["experts"], ld=st["logits"].stride(0))
        st["id"], st["wd"] = qg.layout("i32", t, top_k), qg.layout("f32", t, top_k)
    elif op == "group":
        t, top_k = case["tokens"], case["top_k"]
        st["offsets"] = torch.empty(case["experts"] + 1, device="cuda", dtype=torch.int32)
        st["rows"] = torch.empty(t * top_k, device="cuda", dtype=torch.int32)
        st["back"] = torch.empty(t, top_k, device="cuda", dtype=torch.int32)
        st["id"] = qg.layout("i32", t, top_k)
    elif op in ("quantise", "gated"):
        rows, k, x = case["rows"], case["k"], st["x"]
        st["q"] = torch.empty(rows, up(k, 16), device="cuda", dtype=torch.int8)
        st["s"] = torch.empty(rows, device="cuda")
        st["y"] = torch.empty(rows, up(k, 16 // SIZE[case["dtype"]]), device="cuda", dtype=x.dtype)
        st["xd"] = qg.layout(case["dtype"], x.shape[0], x.shape[1], ld=x.stride(0))
        st["qd"], st["sd"] = qg.layout("i8", rows, k, ld=up(k, 16)), qg.layout("f32", rows, 1)
        st["yd"] = qg.layout(case["dtype"], rows, k, ld=st["y"].stride(0))
        st["act"] = qg.MX_SWIGLU if op == "gated" else qg.MX_IDENTITY
    elif op == "product":
        m, n, k, experts = case["rows"], case["n"], case["k"], case["experts"]
        off, pitch = st["offsets"].data_ptr(), up(n, 8)
        st["d"] = torch.empty(m, pitch, device="cuda", dtype=DT[case["out"]])
        st["op"] = qg.operation(quant_a=(qg.QUANT_BLOCK_F32, 0, 1, 0), quant_b=(qg.QUANT_BLOCK_F32, 0, 1, 0))
        st["ad"], st["ud"] = qg.layout("i8", m, k, ld=up(k, 16), num=experts, offsets=off), qg.layout("f32", m, 1, num=experts, offsets=off)
        st["bd"] = qg.layout("i8", n, k, ld=up(k, 16), num=experts, stride=n * up(k, 16))
        st["vd"] = qg.layout("f32", n, 1, num=experts, stride=n)
        st["dd"] = qg.layout(case["out"], m, n, ld=pitch, num=experts, offsets=off)
        st["cd"] = qg.layout(case["out"], m, n, ld=st["c"].stride(0), num=experts, offsets=off) if case["beta"] else None
    else:
        t, n, k = case["tokens"], case["tokens"] * case["top_k"], case["k"]
        st["y"] = torch.empty(t, up(k, 16 // SIZE[case["out"]]), device="cuda", dtype=DT[case["out"]])
        st["rd"], st["wd"] = qg.layout(case["dtype"], n, k, ld=st["r"].stride(0)), qg.layout("f32", t, case["top_k"])
        st["yd"] = qg.layout(case["out"], t, k, ld=st["y"].stride(0))
        st["cd"] = qg.layout(case["out"], t, k, ld=st["c"].stride(0)) if case["shared"] else None


def run_own(st):
    case = st["case"]
    op = case["op"]
    engine, space = ENGINE
    if op == "route":
        engine.route(st["routing"], st["logits"], st["ld"], st["bias"], st["ids"], st["id"], st["w"], st["wd"])
        return st["ids"], st["w"]
    if op == "group":
        engine.group_rows(case["experts"], st["ids"], st["id"], st["offsets"], st["rows"], st["back"], space.desc)
        return st["offsets"], st["rows"], st["back"]
    if op in ("quantise", "gated"):
        engine.int_quantize(st["x"], st["xd"], st["q"], st["qd"], st["s"], st["sd"], act=st["act"], rows=st.get("index"))
        engine.int_dequantize(st["q"], st["qd"], st["s"], st["sd"], st["y"], st["yd"])
        return st["y"][:, :case["k"]]
    if op == "product":
        engine.run(st["op"], 1.0, st["a"], st["ad"], st["u"], st["ud"], st["b"], st["bd"], st["v"], st["vd"],
                   case["beta"], st["c"], st["cd"], st["d"], st["dd"], space.desc)
        return st["d"][:, :case["n"]]
    engine.combine(st["r"], st["rd"], st["back"], st["w"], st["wd"], st["y"], st["yd"], beta=1.0 if case["shared"] else 0.0, C=st["c"], Cd=st["cd"])
    return st["y"][:, :case["k"]]


# ---- what a pass cannot do without ------------------------------------------------
def work(case):
    op = case["op"]
    if op == "route":
        return {"bytes": case["tokens"] * (case["experts"] * SIZE[case["dtype"]] + 8 * case["top_k"]) + 4 * case["experts"] * case["bias"], "flops": 0}
    if op == "group":
        return {"bytes": 12 * case["tokens"] * case["top_k"] + 4 * case["experts"] + 4, "flops": 0}
    if op == "quantise":
        return {"bytes": (min(case["tokens"], case["rows"]) + case["rows"]) * case["k"] * SIZE[case["dtype"]], "flops": 0}
    if op == "gated":
        return {"bytes": 3 * case["rows"] * case["k"] * SIZE[case["dtype"]], "flops": 0}
    if op == "combine":
        n = case["tokens"] * case["top_k"]
        return {"bytes": int(case["held"] * n) * case["k"] * SIZE[case["dtype"]] + 8 * n + case["tokens"] * case["k"] * SIZE[case["out"]] * (1 + case["shared"]),
                "flops": 2 * case["held"] * n * case["k"]}
    m, n, k, used = case["rows"], case["n"], case["k"], int((counts_of(case) > 0).sum())
    return {"bytes": (m + used * n) * (k + 4) + m * n * SIZE[case["out"]] * (2 if case["beta"] else 1), "flops": 2 * m * n * k}


# ---- from the definition, in 64 bits ------------------------------------------------
def exact_route(st):
    case, x = st["case"], st["logits"].double().cpu().numpy()
    t, e, g = case["tokens"], case["experts"], case["groups"]
    ok = x > -np.inf  # false for NaN too
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            top = np.max(np.where(ok, x, -np.inf), axis=1, keepdims=True)
            p = np.where(ok, np.exp(x - top), 0.0)
            p = np.where(ok, p / np.sum(p, axis=1, keepdims=True), 0.0)
        else:
            p = np.where(ok, np.where(x > 0, 1.0 / (1.0 + np.exp(-x)), np.exp(x) / (1.0 + np.exp(x))), 0.0)
    mark = p + st["bias"].double().cpu().numpy() if case["bias"] else p
    key = np.where(ok, mark if case["bias"] else x, -np.inf)
    if g > 1:
        by_group = np.where(ok, mark, -np.inf).reshape(t, g, e // g)
        if case["group_best"] == 1:
            score = key.reshape(t, g, e // g).max(-1)
        else:
            top = np.sort(by_group, axis=-1)[..., ::-1][..., :2]
            score = np.where(top[..., 0] > -np.inf, np.where(top > -np.inf, top, 0.0).sum(-1), -np.inf)
        rank = np.argsort(np.argsort(-score, axis=-1, kind="stable"), axis=-1, kind="stable")
        key = np.where(np.repeat(rank < case["top_groups"], e // g, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :case["top_k"]]
    live = np.take_along_axis(key, ids, 1) > -np.inf
    w = np.where(live, np.take_along_axis(p, ids, 1), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return torch.from_numpy(np.where(live, ids, -1).astype(np.int32)).cuda(), torch.from_numpy(w * case["scale"]).cuda()


def exact_group(st):
    case, flat = st["case"], st["ids"].cpu().numpy().reshape(-1)
    runs = [np.flatnonzero(flat == e) for e in range(case["experts"])]
    order = np.concatenate(runs)
    rows, back = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    rows[:order.size] = order // case["top_k"]
    back[order] = np.arange(order.size)
    offsets = np.cumsum([0] + [len(r) for r in runs]).astype(np.int32)
    return tuple(torch.from_numpy(x).cuda() for x in (offsets, rows, back.reshape(case["tokens"], -1)))


def nearest(x):
    """x in 64 bits to the int8 grid of its rows: the codes around each value, the nearer one, the even one of two as near."""
    step = (x.abs().max(-1, keepdim=True).values / 127).to(torch.float32).double()
    t = torch.nan_to_num(x / step, nan=0.0, posinf=0.0, neginf=0.0)
    low = torch.floor(t)
    part = t - low
    code = low + ((part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2) == 1))).double()
    return code.clamp(-127, 127) * step


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return exact_route(st)
    if op == "group":
        return exact_group(st)
    if op == "quantise":
        x = st["x"].double()
        return nearest(x if st["index"] is None else x.index_select(0, st["index"].long()))
    if op == "gated":
        x, k = st["x"].double(), case["k"]
        return nearest(torch.sigmoid(x[:, :k]) * x[:, :k] * x[:, k:])
    if op == "combine":
        y = torch.zeros(case["tokens"], case["k"], device="cuda", dtype=torch.float64)
        for j in range(case["top_k"]):
            t = torch.nonzero(st["back"][:, j] >= 0).flatten()
            y.index_add_(0, t, st["w"][t, j, None].double() * st["r"].index_select(0, st["back"][t, j].long()).double())
        return y if st["c"] is None else y + st["c"].double()
    n, k, out, off = case["n"], case["k"], [], st["offsets"].tolist()
    for e in range(case["experts"]):
        a = st["a"][off[e]:off[e + 1], :k].double() * st["u"][off[e]:off[e + 1], None].double()
        b = st["b"][e * n:(e + 1) * n, :k].double() * st["v"][e * n:(e + 1) * n, None].double()
        out.append(torch.mm(a, b.t().contiguous()))
    d = torch.cat(out)
    return d if st["c"] is None else d + case["beta"] * st["c"].double()
