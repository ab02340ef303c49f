"""The operators of an int8 expert block in 64 bits (numpy): int8 rows, the choice of experts, sorting by expert."""
import numpy as np

DT_EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative
DT_TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest step


def up(n, to):
    return -(-n // to) * to


def quantise(y):
    """y (rows x K, float64) -> codes (int8) and scales (float32)."""
    y = np.asarray(y, dtype=np.float64)
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[:, None], 0.0, y)
    amax = np.abs(y).max(-1) if y.shape[1] else np.zeros(len(y))
    with np.errstate(over="ignore"):
        s = (amax / 127.0).astype(np.float32)
    bad |= ~np.isfinite(s)
    s = np.where(bad, np.float32(np.nan), s)
    live = ~bad & (s > 0)
    div = np.where(live, s, 1.0).astype(np.float64)[:, None]
    q = np.where(live[:, None], np.clip(np.rint(y / div), -127, 127), 0.0)  # rint: ties to even
    return q.astype(np.int8), s


def swiglu(x):
    k = x.shape[1] // 2
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return x[:, :k] / (1.0 + np.exp(-x[:, :k])) * x[:, k:]


def route(x, top_k, sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1, renormalize=False, scale=1.0):
    """ids (int32) and weights (float64), one token at a time."""
    x = np.asarray(x, dtype=np.float64)
    t, e = x.shape
    ids, w = np.full((t, top_k), -1, np.int32), np.zeros((t, top_k))
    for i in range(t):
        l = x[i]
        ok = l > -np.inf
        p = np.zeros(e)
        if sigmoid:
            with np.errstate(over="ignore"):
                p[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        elif ok.any():
            top = l[ok].max()
            with np.errstate(invalid="ignore"):
                p[ok] = np.where(l[ok] == top, 1.0, np.exp(l[ok] - top))
            p /= p.sum()
        mark = p + bias if bias is not None else p
        key = mark if bias is not None else l
        ok &= key > -np.inf
        if groups > 1:
            stand = []
            for g in range(groups):
                at = [j for j in range(g * e // groups, (g + 1) * e // groups) if ok[j]]
                if not at:
                    stand.append(-np.inf)
                elif group_best == 1:
                    stand.append(max(key[j] for j in at))
                else:
                    stand.append(sum(sorted((mark[j] for j in at), reverse=True)[:2]))
            best = sorted(range(groups), key=lambda g: (-stand[g], g))[:top_groups]
            ok &= np.isin(np.arange(e) // (e // groups), best)
        order = sorted(np.flatnonzero(ok), key=lambda j: (-key[j], j))[:top_k]
        n = len(order)
        ids[i, :n] = order
        if n and renormalize:
            # as real numbers: logs of the scores over the largest of them
            with np.errstate(invalid="ignore", over="ignore"):
                log = l[order] if not sigmoid else -np.logaddexp(0.0, -l[order])
                r = np.where(log == log.max(), 1.0, np.exp(log - log.max()))
            w[i, :n] = r / r.sum()
        elif n:
            w[i, :n] = p[order]
    return ids, w * scale


def group(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    n, k = flat.size, ids.shape[1]
    rows, back = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    offsets, at = [0], 0
    for e in range(experts):
        for i in np.flatnonzero(flat == e):
            rows[at], back[i] = i // k, at
            at += 1
        offsets.append(at)
    return np.array(offsets, np.int32), rows, back.reshape(ids.shape)
