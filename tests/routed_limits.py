"""Variances of the routed projections' rounding errors, in fp64 (numpy), and
the checks that outputs follow them.

Each rounding is taken as uniform within its half step h and independent of
the others: variance h^2 / 3 (so for weights of either sign, as random ones
are).  Half steps, relative to the value: bf16 2^-8,
fp32 2^-24; an addition inside a matrix instruction is counted with 2^-23, as
if it truncated.  Errors are carried through the products and the activation
to first order (a slot's errors as independent of the token's other slots: an
expert named twice repeats them, which is not modelled).  The model counts,
for y_o = sum_j w_oj x~_j, w = (q - z) d:

- the operand: NS bf16 terms, half step 2^-(8 NS) |x~|; or digits, a scale
  per 32 channels of their largest over 489335 (five) or 7829367 (six digits),
  half step scale / 2, and three fp32 roundings of the largest;
- 4-bit codes in groups of 32 or more, matrix cores: sums P of (16 + q) x~
  (fp32 X: of q minus the zero's integer) per 32 channels in four steps of a
  matrix instruction, groups of more channels growing linearly, their addition
  (times d) to the running sum, which holds up to 128 channels of them, and
  the zero terms;
- digits: the integer sum as fp32 (q - 8 times x~), the zero term, the product;
- other codes: 2 NS products per 32 channels into the running sum;
- the running sum, as large as the terms' root sum of squares R.

An error e has the scale sigma, z = e / sigma.  For n independent values
P(rms(z) > 1 + sqrt(2 t / n)) < exp(-t) (the norm of a Gaussian vector);
t = 12.  One value: |z| <= 7."""
import numpy as np

import oracle
from online_activation_aware_amd import synth
from routed_ref import quantized

U = 2.0 ** -24
M1 = 2.0 ** -23
KMAX = {n: 7 * (16 ** n - 1) // 15 for n in (3, 4, 5, 6)}


class Form:
    """How a call holds x / s and h: NS bf16 terms, or ND digits."""

    def __init__(self, T, bits, group, xt, own=True, wrong=False):
        self.own = own                              # with the operand's own error
        self.wrong = wrong                          # a wrong result: no variance needed
        self.bits, self.group = bits, group
        self.sums = bits == 4 and group >= 32
        self.digits = (5 if xt == "bf16" else 6) if T <= 2 and self.sums else 0
        self.terms = 2 if xt == "bf16" else 3

    def var_operand(self, x):
        """Variance of the operand's own error, x~ [n][K]."""
        v = (U * x) ** 2 / 3                        # the division (or the last product)
        if self.digits:
            top = np.abs(x).reshape(len(x), -1, 32).max(2, keepdims=True) + np.zeros((1, 1, 32))
            return v + ((top / KMAX[self.digits] / 2) ** 2 / 3 + (3 * U * top) ** 2 / 3).reshape(x.shape)
        return v + (2.0 ** (-8 * self.terms) * x) ** 2 / 3

    def round_operand(self, x, less):
        """x~ with `less` terms or digits fewer than the call has."""
        if self.digits:
            top = np.abs(x).reshape(len(x), -1, 32).max(2, keepdims=True)
            sc = np.where(top > 0, top, 1) / KMAX[self.digits - less]
            return (np.rint(x.reshape(len(x), -1, 32) / sc) * sc).reshape(x.shape)
        y, left = np.zeros_like(x), x
        for _ in range(self.terms - less):
            hi = bf16(left)
            y, left = y + hi, left - hi
        return y

    def product(self, x, vx, num, s):
        """(y, variance) of W (x / s); vx: the variance of x."""
        q, d, z = num
        x = x / s
        if self.wrong:
            return x @ ((q - z) * d).T, 0.0
        vx = vx / s ** 2
        w2, x2 = ((q - z) * d) ** 2, x ** 2
        K = x.shape[1]
        R = x2 @ w2.T
        var = (vx + self.own * self.var_operand(x)) @ w2.T
        if self.digits:
            pieces = K / 512 + 1 + 4 + 8 + 16       # of a lane, over lanes, waves and slices
            var += U ** 2 / 3 * (x2 @ ((q - 8) * d).T ** 2 + (3 + pieces) * R)
        elif self.sums:
            per, ng = self.group / 32, 128 / self.group
            if self.terms == 2:
                P, Z = x2 @ (((16 + q) * d) ** 2).T, x2 @ (((16 + z) * d) ** 2).T
            else:
                c = np.rint(z).clip(-128, 128)
                P, Z = x2 @ (((q - c) * d) ** 2).T, x2 @ (((c - z) * d) ** 2).T
            var += M1 ** 2 / 3 * (4 * (per + 1) / 2 * P + 4 * Z) + U ** 2 / 3 * (ng + 1) / 2 * P
            var += R * (U ** 2 / 3 * (K / self.group + 20) + M1 ** 2 / 3 * (K / 32)) / 2
        else:
            var += M1 ** 2 / 3 * (K / 32 * 2 * self.terms * 4 / 2 + 20) * R
        return x @ ((q - z) * d).T, var


# ------------------------------------------------------------------ cases

# Expert layers beside those of the element-wise tests, for what they leave out:
# T, E, topk, K, I, M, bits, group, xt, act, ids
EXPERTS = [
    # the second product in two, two, three and three slices of its channels, the last one shorter, on the matrix cores
    (5, 3, 2, 128, 2336, 40, 4, 32, "bf16", "silu", "any"),
    (7, 3, 2, 128, 2368, 40, 4, 64, "f32", "gelu", "any"),
    (4, 2, 2, 128, 3200, 33, 4, 128, "bf16", "silu", "any"),
    (12, 2, 2, 96, 3200, 40, 4, 32, "f32", "silu", "any"),
    (6, 2, 2, 96, 2336, 40, 3, 16, "f32", "silu", "any"),
    (9, 2, 2, 96, 2112, 40, 2, 32, "bf16", "gelu", "any"),
    (3, 2, 1, 64, 2304, 70, 5, 64, "bf16", "silu", "any"),
    # all tokens on one expert of many: the rows of x~ do not fit and are brought in again
    (16, 8, 1, 2080, 96, 40, 4, 32, "bf16", "silu", "one"),
    (16, 8, 1, 2080, 96, 40, 4, 32, "f32", "gelu", "one"),
    (30, 8, 1, 1152, 2304, 33, 4, 128, "bf16", "silu", "one"),
    (16, 8, 1, 2048, 64, 40, 3, 64, "f32", "silu", "one"),
    # more than 64 experts (the plan's scan in blocks of 64), up to 1024, and up to 32 a token
    (12, 130, 4, 64, 64, 40, 4, 32, "bf16", "silu", "any"),
    (40, 300, 3, 64, 64, 33, 4, 64, "f32", "gelu", "any"),
    (1, 200, 8, 96, 64, 40, 4, 32, "bf16", "silu", "any"),
    (2, 128, 32, 64, 96, 40, 4, 32, "f32", "silu", "any"),
    (3, 1024, 32, 32, 32, 48, 4, 32, "bf16", "silu", "any"),
    (9, 65, 32, 64, 32, 40, 2, 16, "bf16", "gelu", "any"),
    # prompts, to the largest number of tokens
    (700, 5, 3, 96, 64, 33, 4, 32, "bf16", "silu", "any"),
    (1024, 4, 2, 128, 192, 40, 4, 64, "bf16", "gelu", "any"),
    (1024, 70, 4, 64, 32, 32, 3, 32, "f32", "silu", "any"),
]

# Adapters of many tokens in any order, an eighth of the tokens without one: T, K, M, n, rank, xt, at
MIXED = [
    (128, 256, 64, 40, 32, "bf16", "bf16"),
    (200, 4096, 72, 64, 64, "bf16", "bf16"),
    (257, 512, 264, 30, 16, "bf16", "f32"),
    (131, 1032, 136, 200, 8, "bf16", "bf16"),
    (129, 520, 131, 20, 13, "bf16", "bf16"),
    (160, 264, 65, 50, 24, "f32", "bf16"),
    (300, 768, 200, 9, 48, "f32", "f32"),
    (512, 4096, 72, 64, 64, "bf16", "bf16"),
    (600, 1032, 136, 200, 8, "bf16", "bf16"),
    (545, 264, 520, 30, 40, "bf16", "bf16"),
    (530, 2056, 131, 20, 13, "bf16", "bf16"),
    (520, 512, 264, 30, 16, "bf16", "f32"),
    (513, 768, 200, 9, 48, "f32", "f32"),
]

# the same, ids in runs: the last token of every run and tokens without an adapter between them
RUNS = [
    (256, 2048, 192, 5, 64, "bf16", "bf16"),
    (512, 4096, 64, 3, 64, "bf16", "bf16"),
    (700, 3584, 136, 3, 32, "bf16", "f32"),
    (513, 2560, 72, 2, 56, "bf16", "bf16"),
    (515, 128, 48, 2, 40, "f32", "f32"),
    (1000, 512, 264, 9, 16, "bf16", "bf16"),
]


# Shared projections beside those of the element-wise tests: T, K, M, bits, group, n, rank, xt, yt, ids
SHARED = [
    (140, 512, 136, 4, 32, 60, 16, "bf16", "f32", "mixed"),
    (190, 1024, 65, 3, 32, 30, 24, "bf16", "f32", "mixed"),
    (1, 2048, 129, 4, 64, 3, 8, "f32", "f32", "mixed"),
    (4, 1184, 70, 4, 32, 3, 8, "f32", "f32", "mixed"),
    (5, 4096, 40, 4, 128, 6, 16, "f32", "f32", "mixed"),
    (30, 2368, 136, 4, 64, 9, 8, "f32", "f32", "mixed"),
    (140, 3200, 264, 4, 32, 12, 16, "f32", "f32", "mixed"),
    (200, 608, 96, 2, 16, 5, 32, "f32", "f32", "runs"),
    (4200, 128, 64, 4, 32, 5, 8, "f32", "f32", "runs"),
]


def moe_case(case, seed=0):
    """numpy inputs of an expert layer: x (values of its type), ids, w, and
    per weight its codes, steps, zeros, s, and (q, d, z) in fp64."""
    Tn, E, topk, K, I, M, bits, group, xt, act_name, mode = case
    rng = np.random.default_rng(seed + sum(case[:8]))
    x = rng.standard_normal((Tn, K)) * np.where(rng.random(K) < 0.05, 20, 1)
    x = oracle.decode(synth.encode(x, xt), xt)
    ids = np.full((Tn, topk), E - 2) if mode == "one" else rng.integers(0, E, (Tn, topk))
    d = dict(x=x, ids=ids.astype(np.int32), w=(rng.random((Tn, topk)) + 0.1).astype(np.float32))
    for key, rows, cols, per in (("gate_up", 2 * I, K, E % 2 == 0), ("down", M, I, True)):
        codes, step, zero, n = quantized(rng, E, rows, cols, bits, group)
        s = np.exp(rng.standard_normal((E, cols) if per else cols) * 0.5).astype(np.float32)
        d[key] = dict(codes=codes, step=step, zero=zero, s=s, num=n)
    return d


def moe_model(d, case, **kw):
    bits, group, xt, name = case[6:10]
    gu, dn = d["gate_up"], d["down"]
    return moe(d["x"], d["ids"], d["w"].astype(np.float64), gu["num"], gu["s"].astype(np.float64), dn["num"],
               dn["s"].astype(np.float64), bits, name, xt, group, **kw)


def adapter_case(seed, Tn, K, M, n, rank, xt, at, runs=False):
    rng = np.random.default_rng(seed)
    cut = lambda a, t: oracle.decode(synth.encode(a, t), t)   # noqa: E731
    none = rng.random(Tn) < (0.02 if runs else 0.125)
    ids = rng.integers(0, n, Tn)
    ids = np.where(none, -1, np.sort(ids) if runs else ids).astype(np.int32)
    return dict(x=cut(rng.standard_normal((Tn, K)), xt), a=cut(rng.standard_normal((n, rank, K)) / np.sqrt(K), at),
                b=cut(rng.standard_normal((n, M, rank)), at), ids=ids, ranks=rng.integers(0, rank + 1, n).astype(np.int32),
                scale=(rng.random(n) + 0.5).astype(np.float32), rng=rng)


def shared_case(case):
    """Inputs of a shared projection with adapters (a case of the element-wise
    tests; its ids in runs or mixed, at least one token with an adapter of
    full rank), (q, d, z) and s; the packed state under "state"."""
    Tn, K, M, bits, group, n, rank, xt, _, mode = case
    d = adapter_case(sum(case[:7]), Tn, K, M, n, rank, xt, xt)
    rng = d["rng"]
    if mode == "runs":
        d["ids"] = np.sort(rng.integers(0, n, Tn)).astype(np.int32)
    d["ids"][-1], d["ranks"][1] = 1, rank
    codes, step, zero, num = quantized(rng, 1, M, K, bits, group)
    s = np.exp(rng.standard_normal(K) * 0.5).astype(np.float32)
    d["state"] = dict(s=s, codes=codes[0], step=step[0], zero=zero[0])
    return d, tuple(v[0] for v in num), s.astype(np.float64)


# ------------------------------------------------------------------ the model

def bf16(x):
    """Rounded to bf16, to the nearest (ties do not occur in these data)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def act(x, name):
    """(value, slope) of the activation."""
    if name == "silu":
        p = 1 / (1 + np.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def moe(x, ids, wts, gu, s_in, dn, s_down, bits, name, xt, group, less=0, drop_slot=None, drop_channels=0,
        own=True):
    """(Y, variance) of the expert layer.  For wrong results: `less` terms or
    digits fewer, without slot `drop_slot`, or without the last `drop_channels`
    channels of the second product.  own=False: the variance of the sums alone
    (two calls that hold x / s and h alike differ by those)."""
    T, topk = ids.shape
    wrong = bool(less or drop_channels or drop_slot is not None)
    f = Form(T, bits, group, xt, own, wrong)
    E, rows2, _ = gu[0].shape
    I, M = rows2 // 2, dn[0].shape[1]
    y, var = np.zeros((T, M)), np.zeros((T, M))
    at = lambda s, e: s[e] if s.ndim == 2 else s   # noqa: E731
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if drop_slot is not None:
            keep = (t != drop_slot[0]) | (j != drop_slot[1])
            t, j = t[keep], j[keep]
        if len(t) == 0:
            continue
        xe = x[t]
        if less:
            xe = f.round_operand(xe / at(s_in, e), less) * at(s_in, e)
        g, vg = f.product(xe, np.zeros_like(xe), tuple(v[e] for v in gu), at(s_in, e))
        a, da = act(g[:, :I], name)
        u, wt = g[:, I:], wts[t, j][:, None]
        h = a * u * wt
        vh = 0.0 if wrong else (da * u * wt) ** 2 * vg[:, :I] + (a * wt) ** 2 * vg[:, I:] + (h * U) ** 2 / 3 * (8 + (2 * g[:, :I]) ** 2)
        sd = at(s_down, e)
        if less:
            h = f.round_operand(h / sd, less) * sd
        if drop_channels:
            h = np.where(np.arange(I) >= I - drop_channels, 0, h)
        o, vo = f.product(h, vh, tuple(v[e] for v in dn), sd)
        np.add.at(y, t, o)
        np.add.at(var, t, vo + (U * o) ** 2 / 3 * topk)
    return y, var + (U * y) ** 2 / 3


def shared(x, num, s, xt, bits, group):
    """(Y, variance) of the shared projection: for bf16 X, x / s or the
    dequantized weight rounded to bf16; for fp32 X the product of an expert, or
    up to four tokens in fp32 (x times 1 / s, sums per group and lane)."""
    q, d, z = num
    T, K = x.shape
    if xt == "f32" and (T > 4 or K % 128):
        f = Form(3, bits, group, xt)
        y, var = f.product(x, np.zeros_like(x), num, s)
        return y, var + (U * y) ** 2 / 3 * 16      # the slices
    w = (q - z) * d / s
    R = x ** 2 @ (w ** 2).T
    if xt == "f32":                                # fused multiply-adds of q x and sums of x over 32 channels, a lane's groups, 64 lanes
        lane = x ** 2 @ ((q ** 2 + z ** 2) * (d / s) ** 2).T
        return x @ w.T, U ** 2 / 3 * (9 * R + 20 * lane + (K / 32 + 64) * R)
    mag = x ** 2 @ (((q + z + 16) * d / s) ** 2).T
    return x @ w.T, R * 2.0 ** -16 / 3 + M1 ** 2 / 3 * (16 * mag + 4 * K * R)


def adapters(x, A, B, ids, ranks=None, scale=None, f32=False, z_terms=None):
    """(term, variance) of the adapters; z_terms: z cut to so many bf16 terms."""
    T, n = x.shape[0], A.shape[0]
    K, rank = x.shape[1], A.shape[1]
    y = np.zeros((T, B.shape[1]))
    var = np.zeros_like(y)
    for a in range(n):
        t = np.nonzero(ids == a)[0]
        r = rank if ranks is None else int(np.clip(ranks[a], 0, rank))
        if len(t) == 0 or r == 0:
            continue
        sc = 1.0 if scale is None else float(scale[a])
        z = x[t] @ A[a, :r].T
        vz = M1 ** 2 / 3 * ((K if f32 else K / 8) + 16) * (x[t] ** 2 @ (A[a, :r] ** 2).T)
        if z_terms:
            full, left = np.zeros_like(z), z * sc
            for _ in range(z_terms):
                hi = bf16(left)
                full, left = full + hi, left - hi
            z = full / sc
        B2 = (sc * B[a, :, :r]) ** 2
        y[t] = z @ (sc * B[a, :, :r]).T
        var[t] = vz @ B2.T + M1 ** 2 / 3 * ((r if f32 else r / 8) + 12) * (z ** 2 @ B2.T)
    return y, var


def far(got, ref, var, floor=0.0):
    """None, or what is wrong with these outputs."""
    got = np.asarray(got, np.float64)
    if not np.all(np.isfinite(got)):
        return "non-finite outputs"
    sigma = np.sqrt(var + floor ** 2)
    z = np.abs(got - ref) / np.where(sigma > 0, sigma, 1)
    if np.any(z[sigma == 0] != 0):
        return "an output without an error term differs"
    z = np.where(sigma > 0, z, 0)
    if z.max(initial=0.0) > 7:
        return f"an output is off by {z.max():.1f} sigma at {np.unravel_index(z.argmax(), z.shape)}"
    rows = np.sqrt((z ** 2).mean(1))
    if rows.max(initial=0.0) > 1 + np.sqrt(24 / z.shape[1]):
        return f"row {rows.argmax()}: rms {rows.max():.2f} sigma"
    rms = np.sqrt((z ** 2).mean())
    if rms > 1 + np.sqrt(24 / z.size):
        return f"rms {rms:.3f} sigma"
    return None


def check(got, ref, var, floor=0.0):
    wrong = far(got, ref, var, floor)
    assert wrong is None, wrong
