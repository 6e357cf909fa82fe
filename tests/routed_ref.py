"""Definitions in fp64 (numpy) of the projections whose weights each token
chooses, with the element-wise error bounds of the library's arithmetic.

Roundings counted: a bf16 value is off by at most 2^-8 of itself, an fp32 one
by 2^-24.  Inside the matrix products x / s and h are sums of bf16 terms: two
for bf16 X (2^-16), three for fp32 X (2^-24), or fp32 values; codes, steps and
zeros are exact.  Group sums are formed as step (sum (c + q) x - (c + z) sum x)
with c at most 32, so a rounding is relative to step (q + z + 2 c) |x|; a sum
of n terms in fp32 is off by at most n 2^-23 of the sum of the absolute terms
(twice the textbook bound).  One or two tokens on 4-bit codes in groups of 32
or more take x / s and h as integers of five (bf16 X) or six (fp32 X) base-16
digits times a scale per 32 channels: the largest of them is 7 (16^5 - 1) / 15
= 489335 or 7829367 scales, every one is off by half a scale at most, i.e. by
the largest of its 32 over 978670 < 2^-19 or 15658734 < 2^-23, and by another
2^-23 of it for the two roundings before (inverse scale, product)."""
import numpy as np

import oracle

U32 = 2.0 ** -23


def quantized(rng, E, rows, K, bits, group):
    """E random matrices quantized by the oracle: (codes, step, zero) as the
    library stores them, and (q, d, z) as numbers per weight, in fp64."""
    q = np.empty((E, rows, K))
    codes = np.empty((E, rows, K * bits // 32), np.int32)
    step = np.empty((E, rows, K // group), np.float16)
    zero = np.empty_like(step)
    for e in range(E):
        r = oracle.group_rtn((rng.standard_normal((rows, K)) * 0.05).astype(np.float32), bits, group)
        q[e], step[e], zero[e] = r["q"], r["delta"], r["zero"]
        codes[e] = oracle.pack_codes(r["q"], bits)
    num = (q, np.repeat(step.astype(np.float64), group, 2), np.repeat(zero.astype(np.float64), group, 2))
    return codes, step, zero, num


def route(logits, topk, score, renormalize):
    """ids, weights (fp64) and each weight's relative bound."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    T, E = x.shape
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    bound = np.zeros((T, topk))
    for t in range(T):
        order = [e for e in np.argsort(-x[t], kind="stable") if x[t, e] > -np.inf][:topk]
        n = len(order)
        ids[t, :n] = order
        if n == 0:
            continue
        v = x[t, order]
        if score == "softmax":
            m = v[0]
            p = (x[t] == np.inf).astype(np.float64) if m == np.inf else np.exp(x[t] - m)
            p /= p.sum()
            w[t, :n] = p[order]
            # exp: its argument l - m off by 2^-24 of it, itself by 4 roundings; the sum of E terms, the division
            gap = np.where(np.isfinite(v), m - v, 0.0) if m < np.inf else np.zeros(n)
            bound[t, :n] = (np.minimum(gap, 200) + E + 8) * U32
        else:
            with np.errstate(over="ignore"):
                w[t, :n] = 1 / (1 + np.exp(-v))
            bound[t, :n] = (np.where(np.isfinite(v), np.abs(v), 0) + 10) * U32
        if renormalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
            bound[t, :n] = 2 * bound[t, :n].max() + (topk + 4) * U32
    return ids, w, bound


def _gate(x, act):
    if act == "silu":
        return x / (1 + np.exp(-x))
    return 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)))


def _product(x, ex, num, s, bits, rel, digits):
    """y = W (x / s) and a bound on |library - y| where x is off by ex."""
    q, d, z = num
    c = 2.0 ** bits
    w = (q - z) * d / s
    mag = d * (q + z + 2 * c) / s
    K = w.shape[1]
    bound = (np.abs(x) @ mag.T) * (rel + 2.0 ** -21 + K * U32) + ex @ np.abs(w).T
    if digits:
        top = np.repeat((np.abs(x / s) + ex / s).reshape(len(x), K // 32, 32).max(2), 32, axis=1)
        bound += (top @ np.abs(w * s).T) * ((2.0 ** -19 if rel == 2.0 ** -16 else 2.0 ** -23) + U32)
    return x @ w.T, bound


def moe(x, ids, wts, gu, s_in, dn, s_down, bits, act, split, group):
    """gu, dn: (q, d, z) of [E][2 I][K] and [E][M][I]; s_*: [K] or [E][.].
    split: the relative error of x / s and h inside the matrix cores' products.
    Returns (Y, bound)."""
    T = x.shape[0]
    digits = T <= 2 and bits == 4 and group >= 32
    E, rows2, _ = gu[0].shape
    I, M = rows2 // 2, dn[0].shape[1]
    y = np.zeros((T, M))
    by = np.zeros((T, M))
    at = lambda s, e: s[e] if s.ndim == 2 else s   # noqa: E731
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        g, bg = _product(x[t], np.zeros_like(x[t]), tuple(v[e] for v in gu), at(s_in, e), bits, split, digits)
        a = _gate(g[:, :I], act)
        u, bu = g[:, I:], bg[:, I:]
        # |act'| <= 1.2; exp of an argument off by 2^-23 of it, and 8 more roundings
        ba = 1.2 * bg[:, :I] + (np.abs(g[:, :I]) + 8) * 4 * U32 * np.maximum(np.abs(a), np.abs(g[:, :I]) * 1e-3)
        wt = wts[t, j][:, None]
        h = a * u * wt
        bh = ((np.abs(a) + ba) * bu + ba * np.abs(u)) * np.abs(wt) + np.abs(h) * 8 * U32
        o, bo = _product(h, bh, tuple(v[e] for v in dn), at(s_down, e), bits, split, digits)
        np.add.at(y, t, o)
        np.add.at(by, t, bo + np.abs(o) * (ids.shape[1] * U32))
    return y, by


def adapters(x, A, B, ids, ranks=None, scale=None):
    """The adapters' term [T][M] (fp64 A [n][r][K], B [n][M][r]) and its
    bound."""
    T, n = x.shape[0], A.shape[0]
    K, rank = x.shape[1], A.shape[1]
    y = np.zeros((T, B.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        a = int(ids[t])
        if not 0 <= a < n:
            continue
        r = rank if ranks is None else int(np.clip(ranks[a], 0, rank))
        sc = 1.0 if scale is None else float(scale[a])
        y[t] = sc * (B[a, :, :r] @ (A[a, :r] @ x[t]))
        mag[t] = abs(sc) * (np.abs(B[a, :, :r]) @ (np.abs(A[a, :r]) @ np.abs(x[t])))
    return y, mag * ((K + rank + 8) * U32)


def check(got, ref, bound, y_bf16):
    """Every element within its bound plus the output's own rounding."""
    got = np.asarray(got, np.float64)
    lim = bound + np.abs(ref) * (2.0 ** -8 if y_bf16 else 2.0 ** -23) + 1e-30
    lim = lim * (1 + (2.0 ** -7 if y_bf16 else 0.0))   # the rounding of a value that is off by `bound` already
    assert np.all(np.isfinite(got)), "non-finite outputs"
    r = np.abs(got - ref) / lim
    assert float(r.max(initial=0.0)) <= 1.0, \
        f"{int((r > 1).sum())} outputs off (worst ratio {r.max():.3f} at {np.unravel_index(r.argmax(), r.shape)})"
