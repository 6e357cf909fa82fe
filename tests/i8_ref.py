"""Rows in 8 bits, their products and the rows of sorted tokens, on the CPU."""
import numpy as np


def quantize(x, s=None, divide=False):
    """(codes, scales) of the rows of fp64 values that fp32 holds: v and the
    scale in fp32, the quotient in 64 bits (of two 24-bit numbers: its rounding
    is that of the exact quotient)."""
    v = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if s is not None:
            v = v / np.asarray(s, np.float32) if divide else v * np.asarray(s, np.float32)
        top = np.abs(v).max(1)
        scale = top / np.float32(127)
        scale[scale == 0] = 1
        bad = ~np.isfinite(v).all(1)
        q = np.clip(np.rint(v.astype(np.float64) / scale.astype(np.float64)[:, None]), -127, 127)
    q[bad] = 0
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def product(xq, xs, wq, ws):
    """The product in fp32 as it is defined: the exact sum rounded, times the
    two scales, rounded each time."""
    n = xq.astype(np.float64) @ wq.astype(np.float64).T      # whole numbers below 2^53
    with np.errstate(all="ignore"):
        return n.astype(np.float32) * np.asarray(xs, np.float32)[:, None] * np.asarray(ws, np.float32)


def sort(ids, E):
    flat = ids.reshape(-1)
    n = flat.size
    offsets = np.zeros(E + 1, np.int32)
    order, pos = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    r = 0
    for e in range(E):
        for i in np.nonzero(flat == e)[0]:
            order[r], pos[i] = i, r
            r += 1
        offsets[e + 1] = r
    return offsets, order, pos.reshape(ids.shape)


def act(g, name):
    """(act(g), a bound of the error of its fp32 evaluation for a g that is off
    by 3 units of 2^-24): |act'| <= 1.13, so 3.4 |g| of it; the exponential's
    argument has a relative error of 4 units at most (a polynomial of degree
    three for gelu), which times |x| exp(-|x|) <= 0.37 of the argument adds 1.5
    |g|; the exponential, the sum and the quotient 16 units of the value."""
    with np.errstate(over="ignore"):
        if name == "silu":
            a = g / (1 + np.exp(-g))
        else:
            a = g / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    return a, 2.0 ** -24 * (6 * np.abs(g) + 16 * np.abs(a))


def moe(xq, xs, per_slot, ids, w, gu, gu_s, s_down, dn, dn_s, name):
    """(Y, bound) of the layer in fp64.  xq, xs: the codes of X / s_in, [T][K]
    or per_slot [T][topk][K].  bound counts the fp32 roundings and, for each
    code of h whose quotient lies within its error of a border, one step."""
    T, k = ids.shape
    E, rows2, _ = gu.shape
    I, M = rows2 // 2, dn.shape[1]
    u24 = 2.0 ** -24
    y, bound = np.zeros((T, M)), np.zeros((T, M))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0 or e >= E:
                continue
            q, qs = (xq[t, j], xs[t, j]) if per_slot else (xq[t], xs[t])
            gate_up = (gu[e].astype(np.float64) @ q.astype(np.float64)) * float(qs) * gu_s[e].astype(np.float64)
            g, up = gate_up[:I], gate_up[I:]
            a, da = act(g, name)
            sd = (s_down[e] if s_down.ndim == 2 else s_down).astype(np.float64)
            h = a * up / sd
            dh = np.abs(up / sd) * da + 6 * u24 * np.abs(h)      # up: 3 roundings, the product and the quotient 2
            top = np.abs(h).max()
            scale = top / 127 if top > 0 else 1.0
            rel = (dh.max() / top if top > 0 else 0.0) + 4 * u24
            x = h / scale
            code = np.clip(np.rint(x), -127, 127)
            near = np.abs(np.abs(x - np.floor(x)) - 0.5) <= dh / scale + np.abs(x) * rel
            d = dn[e].astype(np.float64)
            out = (d @ code) * scale * dn_s[e]
            step = (np.abs(d) @ near.astype(np.float64)) * scale * dn_s[e]
            y[t] += w[t, j] * out
            bound[t] += abs(w[t, j]) * ((rel + 3 * u24 + (k + 1) * u24) * np.abs(out) + step * (1 + 1e-3))
    return y, bound
