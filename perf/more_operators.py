"""Linear layers in 8-bit integers, and tokens sorted by the experts they chose:

- qgemm: a projection of activations that are quantized per token on the way (ttq_qgemm_i8);
- gemm: the product of codes that are there already, with scales for each token and channel (ttq_gemm_i8);
- dispatch: tokens sorted by expert, and their rows copied in that order (ttq_moe_sort, ttq_moe_gather);
- combine: the experts' rows back in the tokens' order, weighted and added (ttq_moe_combine);
- combine_grad: its gradient, for the rows and for the weights (ttq_moe_combine_grad);
- moe: a gated mixture-of-experts layer of any number of tokens in 8-bit integers (ttq_moe_i8).

A row's 8-bit codes: with a the largest |v| of the row, scale = a / 127 rounded to fp32 (1 where that is 0) and the code
v / scale rounded to the nearest integer, ties to even; v is x / s, rounded to fp32.

`run` makes the library's calls where `own` is true and computes the same with elementary torch operations where it is
false; `exact` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGEST_GEMM = 8192 * 4096 * 4096             # tokens x channels x rows of the largest listed product
LARGEST_ROWS = 8192 * 6 * 2048                # values of the largest listed set of sorted rows
LARGEST_MOE = 2048 * 2 * 4096 * 14336         # token-expert pairs x channels x rows of the largest listed layer


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One new token of one request through a wide-input projection: the stream of the weight is the whole cost.
        dict(name="qgemm_one_token", op="qgemm", T=1, K=14336, M=4096, xt="bf16", yt="bf16"),
        # A prompt through a projection to the wide side of a layer.
        dict(name="qgemm_prompt", op="qgemm", T=2048, K=4096, M=14336, xt="bf16", yt="bf16"),
        # A short prompt on a ragged projection, results in fp32 for what follows.
        dict(name="gemm_ragged_77", op="gemm", T=77, K=2064, M=1411, xt="i8", yt="f32"),
        # Prompts of several requests in one pass, on codes that q, k and v share.
        dict(name="gemm_prompts", op="gemm", T=8192, K=4096, M=4096, xt="i8", yt="bf16"),
        # A step of sixteen requests sent to two of eight experts each: latency alone counts.
        dict(name="dispatch_step_16", op="dispatch", T=16, E=8, topk=2, K=4096, xt="bf16", drop=False),
        # Long prompts over many experts, some of which live elsewhere (slots without an expert).
        dict(name="dispatch_prompt", op="dispatch", T=8192, E=160, topk=6, K=2048, xt="bf16", drop=True),
        # A few tokens of a small model in fp32.
        dict(name="combine_step_5", op="combine", T=5, E=4, topk=2, K=768, xt="f32", yt="f32", drop=True),
        # The way back of the long prompts.
        dict(name="combine_prompt", op="combine", T=8192, E=160, topk=6, K=2048, xt="bf16", yt="bf16", drop=False),
        # A small fine-tuning step in fp32, a quarter of the slots without an expert.
        dict(name="combine_grad_300", op="combine_grad", T=300, E=8, topk=3, K=1056, xt="f32", yt="f32", drop=True),
        # A fine-tuning step over whole sequences.
        dict(name="combine_grad_4096", op="combine_grad", T=4096, E=8, topk=2, K=4096, xt="bf16", yt="bf16", drop=False),
        # A serving step over many small experts of a ragged width, most experts with a handful of tokens.
        dict(name="moe_step_64", op="moe", T=64, E=64, topk=6, K=2048, I=1056, xt="bf16", yt="bf16", act="silu", drop=False),
        # A prompt through two of eight large experts.
        dict(name="moe_prompt", op="moe", T=2048, E=8, topk=2, K=4096, I=14336, xt="bf16", yt="bf16", act="silu", drop=False),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qgemm", "qgemm", "gemm", "gemm", "dispatch", "combine", "combine_grad", "moe", "moe"])
    xt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qgemm", "gemm"):
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), K=16 * _log(rng, 16, 896), M=_log(rng, 200, 14336),
                     xt=xt if op == "qgemm" else "i8", yt=xt)
            if c["T"] * c["K"] * c["M"] <= LARGEST_GEMM:
                return c
    E = _log(rng, 4, 64 if op == "moe" else 256)
    topk = rng.randint(1, min(8, E))
    if op == "moe":
        while True:
            c = dict(op=op, T=_log(rng, 1, 2048), E=E, topk=topk, K=16 * _log(rng, 16, 256), I=16 * _log(rng, 16, 512), xt=xt, yt=xt,
                     act=rng.choice(["silu", "silu", "gelu"]), drop=rng.random() < 0.3)
            if E * c["K"] * c["I"] <= 4 * 4096 * 14336 and c["T"] * topk * c["K"] * c["I"] <= LARGEST_MOE // 4:
                return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 8192), E=E, topk=topk, K=16 * _log(rng, 16, 512), xt=xt, drop=rng.random() < 0.4)
        if op != "dispatch":
            c["yt"] = xt
        if c["T"] * topk * c["K"] * (2 if xt == "f32" else 1) <= LARGEST_ROWS:
            return c


# ------------------------------------------------------------------ inputs

def _codes(v):
    """The 8-bit codes of the rows of v (fp32) and their scales."""
    scale = v.abs().amax(-1) / 127
    scale = torch.where(scale == 0, 1.0, scale)
    # In 64 bits: a quotient next to a border between two codes must not cross it.
    return (v.double() / scale.double()[..., None]).round_().clamp_(-127, 127), scale


def _weights(g, rows, cols, s):
    """Codes and scales of a matrix of N(0, 0.02^2) weights times s."""
    q, scale = _codes(torch.randn((rows, cols), generator=g, device=DEV).mul_(0.02).mul_(s))
    return q.to(torch.int8), scale


def _tokens(g, T, K):
    """Activations with a hundredth of the channels thirty times as large, as layer inputs have them."""
    x = torch.randn((T, K), generator=g, device=DEV)
    return x * torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 30.0, 1.0)


def _scales(g, shape):
    return torch.exp(torch.randn(shape, generator=g, device=DEV) * 0.5)


def _experts(g, c):
    """Each token's experts and weights, as a router gives them; a quarter of the slots empty where slots drop."""
    favour = torch.randn(c["E"], generator=g, device=DEV) * 0.5          # some experts are asked more often
    p = (torch.randn((c["T"], c["E"]), generator=g, device=DEV) + favour).softmax(1)
    w, ids = p.topk(c["topk"], dim=1)
    ids = ids.to(torch.int32)
    if c["drop"]:
        ids = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < 0.25, -1, ids).to(torch.int32)
    return ids.contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    st = {"case": c}
    T, K = c["T"], c["K"]
    if c["op"] in ("qgemm", "gemm"):
        s = _scales(g, (K,))
        st["W"], st["w_scale"] = _weights(g, c["M"], K, s)
        x = _tokens(g, T, K)
        if c["op"] == "qgemm":
            st["X"], st["s"] = x.to(DTYPES[c["xt"]]), s
        else:
            q, st["x_scale"] = _codes(x / s)
            st["X"] = q.to(torch.int8)
        return st
    st["ids"], st["w"] = _experts(g, c)
    if c["op"] == "moe":
        E, I = c["E"], c["I"]
        st["X"] = _tokens(g, T, K).to(DTYPES[c["xt"]])
        for key, rows, cols, s in (("gate_up", 2 * I, K, _scales(g, (K,))), ("down", K, I, _scales(g, (E, I)))):
            q = torch.empty((E, rows, cols), dtype=torch.int8, device=DEV)
            scale = torch.empty((E, rows), device=DEV)
            for e in range(E):
                q[e], scale[e] = _weights(g, rows, cols, s[e] if s.dim() == 2 else s)
            st[key] = {"s": s, "codes": q, "scale": scale}
        return st
    n = T * c["topk"]
    xt = DTYPES[c["xt"]]
    if c["op"] == "dispatch":
        st["X"] = _tokens(g, T, K).to(xt)
        st["R"] = torch.zeros((n, K), dtype=xt, device=DEV)       # rows behind the last one stay as they were
        return st
    st["pos"] = _sort(st["ids"], c["E"])[2]
    st["R"] = torch.randn((n, K), generator=g, device=DEV).to(xt)
    if c["op"] == "combine_grad":
        st["dY"] = torch.randn((T, K), generator=g, device=DEV).to(DTYPES[c["yt"]])
        st["dR"] = torch.zeros((n, K), dtype=xt, device=DEV)
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    from online_activation_aware_amd import ttq
    c = st["case"]
    op, T, K = c["op"], c["T"], c["K"]
    if op == "combine":
        return ttq.ttq_moe_combine(st["R"], st["pos"], st["w"], y_dtype=DTYPES[c["yt"]])
    if op == "combine_grad":
        return list(ttq.ttq_moe_combine_grad(st["dY"], st["R"], st["pos"], st["w"], dR=st["dR"]))
    if "ws" not in st:    # a program keeps its workspace
        st["ws"] = (ttq.qgemm_i8_workspace(T, K, c["M"]) if op == "qgemm" else ttq.gemm_i8_workspace(T, K, c["M"]) if op == "gemm" else
                    ttq.moe_sort_workspace(T, c["topk"], c["E"]) if op == "dispatch" else
                    ttq.moe_i8_workspace(T, c["topk"], K, c["I"], K, c["E"]))
    if op == "qgemm":
        return ttq.ttq_qgemm_i8(st["X"], st["s"], st["W"], st["w_scale"], y_dtype=DTYPES[c["yt"]], ws=st["ws"])
    if op == "gemm":
        return ttq.ttq_gemm_i8(st["X"], st["x_scale"], st["W"], st["w_scale"], y_dtype=DTYPES[c["yt"]], ws=st["ws"])
    if op == "dispatch":
        offsets, order, pos = ttq.ttq_moe_sort(st["ids"], c["E"], ws=st["ws"])
        return [offsets, order, pos, ttq.ttq_moe_gather(st["X"], pos, R=st["R"])]
    return ttq.ttq_moe_i8(st["X"], st["ids"], st["w"], st["gate_up"], st["down"], act=c["act"], y_dtype=DTYPES[c["yt"]], ws=st["ws"])


def _sort(ids, E):
    """offsets [E + 1], order [slots] (-1 behind the last row) and pos [T][topk] (-1 without an expert) of a stable sort."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    by = torch.sort(key, stable=True)
    offsets = (key[:, None] < torch.arange(E + 1, device=DEV)).sum(0).to(torch.int32)
    at = torch.arange(n, device=DEV)
    order = torch.where(by.values < E, by.indices, -1).to(torch.int32)
    pos = torch.empty(n, dtype=torch.int32, device=DEV)
    pos[by.indices] = torch.where(by.values < E, at, -1).to(torch.int32)
    return offsets, order, pos.view(ids.shape)


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
    return x * (1 - 1 / (1 + torch.exp(2 * u)))     # x (1 + tanh u) / 2


def _product(q, scale, W, w_scale):
    """Rows of codes (as fp32) times the rows of W (8-bit codes), scaled, in fp32."""
    return (q @ W.float().T) * scale[:, None] * w_scale


def _plain(st):
    c = st["case"]
    op, T = c["op"], c["T"]
    if op == "qgemm":
        q, scale = _codes(st["X"].float() / st["s"])
        return _product(q.float(), scale, st["W"], st["w_scale"]).to(DTYPES[c["yt"]])
    if op == "gemm":
        return _product(st["X"].float(), st["x_scale"], st["W"], st["w_scale"]).to(DTYPES[c["yt"]])
    k = c["topk"]
    if op == "dispatch":
        offsets, order, pos = _sort(st["ids"], c["E"])
        st["R"].copy_(torch.where((order >= 0)[:, None], st["X"][order.long().clamp(min=0) // k], st["R"]))
        return [offsets, order, pos, st["R"]]
    if op == "moe":
        return _plain_moe(st).to(DTYPES[c["yt"]])
    pos = st["pos"].long()
    have = (pos >= 0)[..., None]
    if op == "combine":
        rows = torch.where(have, st["R"][pos.clamp(min=0)].float() * st["w"][..., None], 0.0)
        return rows.sum(1).to(DTYPES[c["yt"]])
    dY = st["dY"].float()
    dw = torch.where(have, st["R"][pos.clamp(min=0)].float() * dY[:, None], 0.0).sum(2)
    at = torch.where(pos >= 0, pos, T * k).reshape(-1)           # slots without a row land behind the rows
    dR = torch.cat((st["dR"], st["dR"][:1]))
    dR[at] = (dY[:, None] * st["w"][..., None]).reshape(T * k, -1).to(dR.dtype)
    st["dR"].copy_(dR[:-1])
    return [st["dR"], dw]


def _plain_moe(st):
    c = st["case"]
    T, E, I, k = c["T"], c["E"], c["I"], c["topk"]
    gu, dn, w = st["gate_up"], st["down"], st["w"]
    ids = st["ids"].long()
    q, scale = _codes(st["X"].float() / gu["s"])
    q = q.float()

    def hidden(g, s):
        h, hs = _codes(_act(g[..., :I], c["act"]) * g[..., I:] / s)
        return h.float(), hs
    if T <= 64:      # every expert for every token, weighted by the token's share of it
        share = torch.zeros((T, E), device=DEV).scatter_add_(1, ids.clamp(min=0), torch.where(ids < 0, 0.0, w))
        g = (q @ gu["codes"].view(E * 2 * I, -1).float().T).view(T, E, 2 * I).transpose(0, 1)
        h, hs = hidden(g * scale[:, None] * gu["scale"][:, None], dn["s"][:, None])
        y = torch.matmul(h, dn["codes"].float().transpose(1, 2).contiguous())
        return (y * hs[..., None] * dn["scale"][:, None] * share.T[..., None]).sum(0)
    offsets, order, pos = _sort(st["ids"], E)
    order = order.long()
    rows = torch.zeros((T * k + 1, c["K"]), device=DEV)          # the last row stays zero, for slots without an expert
    at = offsets.tolist()
    for e in range(E):
        t = order[at[e]:at[e + 1]] // k
        if at[e] < at[e + 1]:
            h, hs = hidden(_product(q[t], scale[t], gu["codes"][e], gu["scale"][e]), dn["s"][e])
            rows[at[e]:at[e + 1]] = _product(h, hs, dn["codes"][e], dn["scale"][e])
    return (rows[pos.long()] * w[..., None]).sum(1)


# ------------------------------------------------------------------ the definitions in 64 bits

def _rows64(v):
    """The 8-bit values of the rows of v (fp64), as codes and the scales in fp32's precision."""
    top = v.abs().max(dim=1).values
    scale = (top / 127).float().double()
    scale[scale == 0] = 1
    return torch.clamp(torch.round(v / scale[:, None]), -127, 127), scale


def _matmul64(a, b):
    """a b^T in fp64, a block of b's rows at a time."""
    return torch.cat([a @ part.double().T for part in b.split(2048)], dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    T, K = c["T"], c["K"]
    if c["op"] in ("qgemm", "gemm"):
        if c["op"] == "qgemm":
            q, scale = _rows64((st["X"].double() / st["s"].double()).float().double())
        else:
            q, scale = st["X"].double(), st["x_scale"].double()
        return _matmul64(q, st["W"]) * scale[:, None] * st["w_scale"].double()
    ids = st["ids"].reshape(-1)
    k = c["topk"]
    if c["op"] == "dispatch":
        lists = [torch.nonzero(ids == e)[:, 0] for e in range(c["E"])]
        order = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
        rows = torch.cat(lists)
        order[:rows.numel()] = rows.to(torch.int32)
        pos = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
        pos[rows] = torch.arange(rows.numel(), dtype=torch.int32, device=DEV)
        offsets = torch.zeros(c["E"] + 1, dtype=torch.int32)
        offsets[1:] = torch.tensor([len(i) for i in lists]).cumsum(0)
        R = torch.zeros((T * k, K), dtype=torch.float64, device=DEV)
        R[:rows.numel()] = st["X"].double().repeat_interleave(k, 0)[rows]
        return [offsets.to(DEV), order, pos.view(T, k), R]
    if c["op"] == "moe":
        y = torch.zeros((T, K), dtype=torch.float64, device=DEV)
        gu, dn = st["gate_up"], st["down"]
        q, scale = _rows64((st["X"].double() / gu["s"].double()).float().double())
        for e in range(c["E"]):
            t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
            if t.numel() == 0:
                continue
            g = _matmul64(q[t], gu["codes"][e]) * scale[t][:, None] * gu["scale"][e].double()
            g, u = g[:, :c["I"]], g[:, c["I"]:]
            if c["act"] == "silu":
                a = g * torch.special.expit(g)
            else:
                a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
            h, hs = _rows64(a * u / dn["s"][e].double())
            out = _matmul64(h, dn["codes"][e]) * hs[:, None] * dn["scale"][e].double()
            y.index_add_(0, t, out * st["w"].double()[t, j][:, None])
        return y
    slot = torch.nonzero(st["pos"].reshape(-1) >= 0)[:, 0]       # slots that have a row
    row, token, w = st["pos"].reshape(-1)[slot].long(), slot // k, st["w"].double().reshape(-1)[slot]
    if c["op"] == "combine":
        y = torch.zeros((T, K), dtype=torch.float64, device=DEV)
        return y.index_add_(0, token, st["R"].double()[row] * w[:, None])
    dY = st["dY"].double()
    dR = torch.zeros((T * k, K), dtype=torch.float64, device=DEV)
    dR[row] = dY[token] * w[:, None]
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[slot] = (dY[token] * st["R"].double()[row]).sum(1)
    return [dR, dw.view(T, k)]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    T, K = c["T"], c["K"]
    size = {"f32": 4, "bf16": 2, "i8": 1}
    if c["op"] in ("qgemm", "gemm"):
        M = c["M"]
        side = 4 * K if c["op"] == "qgemm" else 4 * T
        return {"bytes": T * K * size[c["xt"]] + M * K + 4 * M + side + T * M * size[c["yt"]], "flops": 2 * T * M * K}
    pairs = T * c["topk"] * (0.75 if c["drop"] else 1)
    slots = 4 * T * c["topk"]
    row = K * size[c["xt"]]
    if c["op"] == "dispatch":
        return {"bytes": slots * 3 + 4 * (c["E"] + 1) + T * row + pairs * row, "flops": 0}
    if c["op"] == "combine":
        return {"bytes": slots * 2 + pairs * row + T * K * size[c["yt"]], "flops": 2 * pairs * K}
    if c["op"] == "combine_grad":
        return {"bytes": slots * 3 + 2 * pairs * row + T * K * size[c["yt"]], "flops": 3 * pairs * K}
    experts = c["E"] * (1 - (1 - c["topk"] / c["E"]) ** T) * (1 if T > 8 or not c["drop"] else 0.75)   # distinct ones, as many as are expected
    return {"bytes": experts * (3 * K * c["I"] + 4 * (2 * c["I"] + K)) + T * K * (size[c["xt"]] + size[c["yt"]]) + slots * 2,
            "flops": 6 * pairs * K * c["I"]}
