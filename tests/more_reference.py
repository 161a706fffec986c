"""Plain 64-bit references of routing, its gradient and the MX-FP4 format (no tests here).

Bounds of routing, in fp32 steps of 2^-23 relative.  exp of an argument x: the subtraction
that made x is off by |x| 2^-24, the product with log2 e by as much again of its constant
(what the rounding of the product takes is put back), the hardware's exp2 and
the multiplication by one step each: (2 + |x|) steps.  A sigmoid adds the sum 1 + exp,
half a step, and a reciprocal, one: (4 + |x|).  A sum of E terms adds E half steps, a
quotient one, the scale one.
"""
import numpy as np

F32 = 2.0 ** -23
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E2M1 = np.concatenate([E2M1, -E2M1])


def scores(l, kind):
    """float64 [N, E]; a row of -inf gives zeros under softmax, a NaN its whole row."""
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-l))
        out = np.zeros_like(l)
        for t, row in enumerate(l):
            if np.isnan(row).any() or np.isposinf(row).any():
                out[t] = np.nan
            elif np.isfinite(row).any():
                e = np.exp(row - row.max())
                out[t] = e / e.sum()
        return out


def _better(v):
    """Sort key: larger first, a NaN before all."""
    return (0, 0.0) if np.isnan(v) else (1, -v)


def choose(l, bias, r, k):
    """IDs [N, k] by the definition, a token at a time; r: the router's fields as a dict."""
    l = np.asarray(l, dtype=np.float64)
    n, e = l.shape
    s = scores(l, r["score"])
    groups, each = r.get("n_groups", 1), e // r.get("n_groups", 1)
    ids = np.full((n, k), -1, dtype=np.int32)
    for t in range(n):
        biased = s[t] + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        key = l[t] if bias is None else biased
        ok = [i for i in range(e) if not np.isneginf(l[t, i]) and not np.isneginf(key[i])]
        if r.get("top_groups", 1) < groups:
            part = biased if r.get("group_top", 1) == 2 else key
            total = []
            for q in range(groups):
                best = sorted((part[i] for i in ok if i // each == q and not np.isneginf(part[i])), key=_better)
                best = best[: r.get("group_top", 1)]
                if best:
                    total.append((_better(sum(best)), q))
            kept = {q for _, q in sorted(total)[: r["top_groups"]]}
            ok = [i for i in ok if i // each in kept]
        ok.sort(key=lambda i: (_better(key[i]), i))
        ids[t, : len(ok[:k])] = ok[:k]
    return ids


def gates(l, ids, r):
    """(weights [N, k], bound) of given IDs."""
    l = np.asarray(l, dtype=np.float64)
    s = scores(l, r["score"])
    rows = np.arange(len(l))[:, None]
    live = ids >= 0
    with np.errstate(all="ignore"):
        v = np.where(live, s[rows, ids], 0.0)
        # the arguments of the exponentials behind each weight and behind its sum
        arg = np.abs(np.where(live, l[rows, ids], 0.0))
        if r["score"] == "softmax":
            top = np.where(np.isneginf(l).all(1), 0.0, np.nanmax(np.where(np.isneginf(l), -1e300, l), axis=1))
            arg = np.abs(np.where(live, l[rows, ids] - top[:, None], 0.0))
        steps = arg + arg.max(axis=1, keepdims=True, initial=0) + 10 + l.shape[1]
        if r.get("renormalize", True):
            if r["score"] == "softmax":  # of the chosen logits alone: no underflow of the whole row's
                c = np.where(live, l[rows, ids], -np.inf)
                m = c.max(axis=1, keepdims=True, initial=-np.inf)
                v = np.where(live, np.exp(c - np.where(np.isneginf(m), 0.0, m)), 0.0)
                v = np.where(np.isnan(s).any(1, keepdims=True) & live, np.nan, v)
            total = v.sum(axis=1, keepdims=True)
            v = np.where(live, v / np.where(total == 0, 1, total), 0.0)
        w = v * r.get("scale", 1.0)
        return w, steps * F32 * np.abs(w) + 2.0 ** -125 * abs(r.get("scale", 1.0))


def route_gradient(l, ids, dweights, dscores, r):
    """(dlogits, bound before its rounding)."""
    l = np.asarray(l, dtype=np.float64)
    n, e = l.shape
    s = scores(l, r["score"])
    rows = np.arange(n)[:, None]
    live = (ids >= 0) & (ids < e)
    at = np.where(live, ids, 0)
    scale = r.get("scale", 1.0)
    direct, d = np.zeros((n, e)), np.zeros((n, e)) if dscores is None else np.asarray(dscores, dtype=np.float64).copy()
    m_direct, m = np.zeros((n, e)), np.abs(d)
    if dweights is not None:
        u = np.where(live, np.asarray(dweights, dtype=np.float64), 0.0) * scale
        if r.get("renormalize", True):
            w = gates(l, np.where(live, ids, -1), dict(r, scale=1.0))[0]
            mag = w * (np.abs(u) + (np.abs(u) * w).sum(1, keepdims=True))
            u = w * (u - (u * w).sum(1, keepdims=True))
            if r["score"] == "sigmoid":
                # 1 - s loses what s is off: a step of 1
                u, mag = u * (1 - s[rows, at]), mag
            np.add.at(direct, (np.broadcast_to(rows, at.shape), at), np.where(live, u, 0))
            np.add.at(m_direct, (np.broadcast_to(rows, at.shape), at), np.where(live, mag, 0))
        else:
            np.add.at(d, (np.broadcast_to(rows, at.shape), at), u)
            np.add.at(m, (np.broadcast_to(rows, at.shape), at), np.abs(u))
    if r["score"] == "sigmoid":
        dl, mag = direct + d * s * (1 - s), m_direct + m * s
    else:
        dl = direct + s * (d - (d * s).sum(1, keepdims=True))
        mag = m_direct + s * (m + (m * s).sum(1, keepdims=True))
    arg = np.abs(np.where(np.isfinite(l), l, 0)).max(axis=1, keepdims=True, initial=0) * 2
    return dl, (3 * arg + 2 * e + 40) * F32 * mag + 1e-37


# ---- MX-FP4 -------------------------------------------------------------------------


def mx_value(codes, scales):
    """float64 values of uint8 codes [.., C/2] and scale bytes [.., C/32]; byte 255: NaN."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], -1)
    x = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(x, 32, axis=-1)


def mx_encode(v):
    """(codes, scale bytes) of float64 values [.., C], a block at a time by the definition."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(-1, 32)
    codes, scales = np.zeros(b.shape, dtype=np.uint8), np.zeros(len(b), dtype=np.uint8)
    for i, block in enumerate(b):
        top = np.abs(block).max()
        if not np.isfinite(top):
            scales[i] = 255
            continue
        x = -127 if top == 0 else max(np.frexp(top)[1] - 1 - 2, -127)
        scales[i] = x + 127
        a = np.abs(np.ldexp(block, -x))
        near = np.abs(a[:, None] - E2M1[None, :8])
        # of two equally near the even code
        code = np.array([min(range(8), key=lambda c: (near[j, c], c & 1)) for j in range(32)])
        codes[i] = code + 8 * np.signbit(block)
    codes = codes.reshape(*v.shape[:-1], -1, 2)
    return (codes[..., 0] | codes[..., 1] << 4).astype(np.uint8), scales.reshape(*v.shape[:-1], -1)
