"""Projections whose weights each token chooses, beside the quantized projections of one layer:

- route: the top-k experts and their weights from a token's router logits (ttq_moe_route);
- moe: a gated mixture-of-experts layer on quantized experts, for few tokens (ttq_moe);
- adapters: low-rank adapters of many requests added to a projection (ttq_adapters_add);
- shared: a quantized projection shared by the requests, plus their adapters (ttq_qgemm_adapters).

`run` makes the library's calls where `own` is true and computes the same with elementary torch operations
where it is false; `exact` evaluates the definitions in 64 bits, expert by expert and adapter by adapter.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGEST_MOE = 128 * 2 * 4096 * 14336          # token-expert pairs x channels x rows of the largest listed layer


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One new token of one request: the router of a layer with eight experts.  Latency alone counts.
        dict(name="route_one_token", op="route", T=1, E=8, topk=2, lt="f32", score="softmax", renorm=True, masked=False),
        # A long prompt, many experts, sigmoid scores, with experts that are masked off for some tokens.
        dict(name="route_prompt", op="route", T=8192, E=160, topk=6, lt="bf16", score="sigmoid", renorm=True, masked=True),
        # One new token through two of eight large experts: the stream of their codes is the whole cost.
        dict(name="moe_one_token", op="moe", T=1, E=8, topk=2, K=4096, I=14336, bits=4, group=32, xt="bf16", yt="bf16", act="silu", drop=False),
        # A step of sixteen requests over many small experts of a ragged width, most experts with a token or two.
        dict(name="moe_step_16", op="moe", T=16, E=64, topk=6, K=2048, I=1056, bits=4, group=32, xt="bf16", yt="bf16", act="silu", drop=False),
        # A small model in fp32 with 3-bit codes in groups of 16; some experts live elsewhere (slots without an expert).
        dict(name="moe_small_f32", op="moe", T=5, E=4, topk=2, K=768, I=2048, bits=3, group=16, xt="f32", yt="f32", act="gelu", drop=True),
        # A busy serving step: every expert has tens of tokens.
        dict(name="moe_step_128", op="moe", T=128, E=8, topk=2, K=4096, I=14336, bits=4, group=64, xt="bf16", yt="bf16", act="silu", drop=False),
        # One request's step beside a square projection.
        dict(name="adapters_one_token", op="adapters", T=1, K=4096, M=4096, L=8, R=16, ragged=False, segments=0, none=False, xt="bf16", at="bf16", yt="bf16"),
        # A step of 48 requests with adapters of their own and ranks up to 32, an eighth of them without one.
        dict(name="adapters_step_48", op="adapters", T=48, K=4096, M=14336, L=64, R=32, ragged=True, segments=0, none=True, xt="bf16", at="bf16", yt="bf16"),
        # Prompts of five requests in one pass, each a run of tokens.
        dict(name="adapters_prompts", op="adapters", T=2048, K=4096, M=4096, L=8, R=64, ragged=True, segments=5, none=False, xt="bf16", at="bf16", yt="bf16"),
        # Four requests' step through a wide-input projection.
        dict(name="shared_step_4", op="shared", T=4, K=14336, M=4096, bits=4, group=32, L=16, R=16, ragged=False, segments=0, none=False, xt="bf16", at="bf16", yt="bf16"),
        # Sixteen requests' step through a square projection.
        dict(name="shared_step_16", op="shared", T=16, K=4096, M=4096, bits=4, group=32, L=32, R=16, ragged=True, segments=0, none=True, xt="bf16", at="bf16", yt="bf16"),
        # Prompts of three requests through a square projection.
        dict(name="shared_prompts", op="shared", T=1024, K=4096, M=4096, bits=4, group=32, L=8, R=32, ragged=False, segments=3, none=False, xt="bf16", at="bf16", yt="bf16"),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "adapters", "adapters", "shared", "shared"])
    if op == "route":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, topk=rng.randint(1, min(8, E)), lt=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5, masked=rng.random() < 0.5)
    bits = rng.choice([4, 4, 4, 4, 2, 3, 5])
    group = rng.choice([32, 32, 64, 128, 16])
    unit = max(32, group)
    xt = rng.choice(["bf16", "bf16", "f32"])
    if op == "moe":
        while True:
            E = _log(rng, 4, 64)
            c = dict(op=op, T=_log(rng, 1, 128), E=E, topk=rng.randint(1, min(6, E)), K=unit * _log(rng, 256 // unit, 4096 // unit),
                     I=unit * _log(rng, 256 // unit, 8192 // unit), bits=bits, group=group, xt=xt, yt=xt, act=rng.choice(["silu", "silu", "gelu"]),
                     drop=rng.random() < 0.3)
            if E * c["K"] * c["I"] <= 4 * 4096 * 14336 and c["T"] * c["topk"] * c["K"] * c["I"] <= LARGEST_MOE // 4:
                return c
    c = dict(op=op, T=_log(rng, 1, 2048 if op == "adapters" else 1024), K=unit * _log(rng, 256 // unit, 8192 // unit), M=_log(rng, 200, 8192),
             L=_log(rng, 1, 64), R=_log(rng, 1, 64), ragged=rng.random() < 0.5, segments=0, none=rng.random() < 0.3, xt=xt,
             at=rng.choice(["bf16", "bf16", "f32"]), yt=xt)
    if c["T"] > 64:
        c["segments"] = rng.randint(1, 9)
    if op == "shared":
        c.update(bits=bits, group=group)
    # No more work than the largest listed layer, and tables of adapters that fit the card easily.
    while c["L"] * c["R"] * (c["K"] + c["M"]) > 1 << 27:
        c["L"] = max(1, c["L"] // 2)
    return c


# ------------------------------------------------------------------ inputs

def _quantize(w, bits, group):
    """Asymmetric round-to-nearest codes of w [rows][cols] (fp32): int32 words (code j of a row in bits
    [bits j, bits j + bits) of its little-endian stream), fp16 steps and fp16 integer zeros per group."""
    rows, cols = w.shape
    v = w.view(rows, cols // group, group)
    lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
    top = (1 << bits) - 1
    step = ((hi - lo) / top).to(torch.float16).clamp(min=1e-6)
    sf = step.float()
    zero = (-lo / sf).round().clamp(0, top)
    q = ((v / sf[..., None]).round() + zero[..., None]).clamp(0, top).to(torch.int32).view(rows, cols // 32, 32)
    bit = (q[..., None] >> torch.arange(bits, device=w.device, dtype=torch.int32)) & 1
    bit = bit.view(rows, cols // 32, bits, 32) << torch.arange(32, device=w.device, dtype=torch.int32)
    words = bit.sum(3, dtype=torch.int32).view(rows, cols * bits // 32)
    return words, step, zero.to(torch.float16)


def _state(g, n, rows, cols, bits, group, s):
    """Quantized state of n matrices [rows][cols] of N(0, 0.02^2) weights times s (an [n][cols] or [cols] vector)."""
    codes = torch.empty((n, rows, cols * bits // 32), dtype=torch.int32, device=DEV)
    step = torch.empty((n, rows, cols // group), dtype=torch.float16, device=DEV)
    zero = torch.empty_like(step)
    for e in range(n):
        w = torch.randn((rows, cols), generator=g, device=DEV) * 0.02 * (s[e] if s.dim() == 2 else s)
        codes[e], step[e], zero[e] = _quantize(w, bits, group)
    return {"s": s, "codes": codes, "scale_f16": step, "zero_f16": zero}


def _tokens(g, T, K, dtype):
    """Activations with a hundredth of the channels thirty times as large, as layer inputs have them."""
    x = torch.randn((T, K), generator=g, device=DEV)
    x *= torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 30.0, 1.0)
    return x.to(DTYPES[dtype])


def _scales(g, shape):
    return torch.exp(torch.randn(shape, generator=g, device=DEV) * 0.5)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    st = {"case": c}
    T = c["T"]
    if c["op"] == "route":
        x = torch.randn((T, c["E"]), generator=g, device=DEV) * 2.0
        if c["masked"]:   # experts masked off for some tokens; a few tokens have none left
            off = torch.rand((T, c["E"]), generator=g, device=DEV) < 0.2
            off |= torch.rand((T, 1), generator=g, device=DEV) < 0.01
            x = x.masked_fill(off, -math.inf)
        st["logits"] = x.to(DTYPES[c["lt"]])
        return st
    st["X"] = _tokens(g, T, c["K"], c["xt"])
    if c["op"] == "moe":
        E, K, I = c["E"], c["K"], c["I"]
        p = torch.randn((T, E), generator=g, device=DEV).softmax(1)
        w, ids = p.topk(c["topk"], dim=1)
        ids = ids.to(torch.int32)
        if c["drop"]:
            ids = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < 0.25, -1, ids).to(torch.int32)
        st["ids"], st["w"] = ids.contiguous(), (w / w.sum(1, keepdim=True)).contiguous()
        st["gate_up"] = _state(g, E, 2 * I, K, c["bits"], c["group"], _scales(g, (K,)))
        st["down"] = _state(g, E, K, I, c["bits"], c["group"], _scales(g, (E, I)))
        return st
    K, M, L, R = c["K"], c["M"], c["L"], c["R"]
    at = DTYPES[c["at"]]
    st["A"] = (torch.randn((L, R, K), generator=g, device=DEV) / math.sqrt(K)).to(at)
    st["B"] = (torch.randn((L, M, R), generator=g, device=DEV) * 0.3).to(at)
    st["scale"] = torch.rand(L, generator=g, device=DEV) + 0.5
    st["ranks"] = torch.randint(1, R + 1, (L,), generator=g, device=DEV, dtype=torch.int32) if c["ragged"] else None
    if c["segments"]:   # runs of tokens, one adapter each
        cuts = torch.sort(torch.randint(0, T, (c["segments"] - 1,), generator=g, device=DEV)).values
        run_of = torch.searchsorted(cuts, torch.arange(T, device=DEV), right=True)
        ids = torch.randint(0, L, (c["segments"],), generator=g, device=DEV)[run_of]
    else:               # one token a request, adapters as they come
        ids = torch.randperm(max(L, T), generator=g, device=DEV)[:T] % L
    if c["none"]:
        ids = torch.where(torch.rand(T, generator=g, device=DEV) < 0.125, -1, ids)
    st["ids"] = ids.to(torch.int32).contiguous()
    if c["op"] == "adapters":
        st["C"] = torch.randn((T, M), generator=g, device=DEV).to(DTYPES[c["yt"]])
    else:
        s = _state(g, 1, M, K, c["bits"], c["group"], _scales(g, (K,)))
        st["state"] = {"s": s["s"], **{k: s[k][0] for k in ("codes", "scale_f16", "zero_f16")}}
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    from online_activation_aware_amd import ttq
    c = st["case"]
    if c["op"] == "route":
        return list(ttq.ttq_moe_route(st["logits"], c["topk"], score=c["score"], renormalize=c["renorm"]))
    X, yt = st["X"], DTYPES[c["yt"]]
    if c["op"] == "moe":
        if "ws" not in st:    # a program keeps its workspace
            st["ws"] = ttq.moe_workspace(c["T"], c["topk"], c["K"], c["I"], c["K"], c["E"], c["bits"], c["group"], device=X.device)
        return ttq.ttq_moe(X, st["ids"], st["w"], st["gate_up"], st["down"], c["bits"], c["group"], act=c["act"], y_dtype=yt, ws=st["ws"])
    if c["op"] == "adapters":
        if "ws" not in st:
            st["ws"] = ttq.adapters_workspace(c["T"], c["K"], c["M"], c["R"], device=X.device)
        return ttq.ttq_adapters_add(X, st["A"], st["B"], st["ids"], C=st["C"], ranks=st["ranks"], scale=st["scale"], y_dtype=yt, ws=st["ws"])
    q = st["state"]
    if "ws" not in st:
        st["ws"] = ttq.qgemm_adapters_workspace(c["T"], c["K"], c["M"], c["bits"], c["group"], c["R"], device=X.device)
    return ttq.ttq_qgemm_adapters(X, q["s"], q["codes"], q["scale_f16"], q["zero_f16"], c["M"], c["bits"], c["group"], st["A"], st["B"], st["ids"],
                                  ranks=st["ranks"], scale=st["scale"], y_dtype=yt, ws=st["ws"])


def _codes(words, bits):
    """The codes of packed rows, as small integers."""
    if bits == 4:
        b = words.view(torch.uint8)
        return torch.stack((b & 15, b >> 4), -1).flatten(-2)
    w = words.view(*words.shape[:-1], -1, bits).to(torch.int64) & 0xFFFFFFFF
    at = torch.arange(32, device=words.device) * bits
    lo = w[..., at >> 5]
    hi = w[..., ((at >> 5) + 1).clamp(max=bits - 1)]
    return ((((hi << 32) | lo) >> (at & 31)) & ((1 << bits) - 1)).flatten(-2).to(torch.uint8)


def _weights(codes, step, zero, bits, group):
    """(code - zero) step in fp32."""
    q = _codes(codes, bits).float().unflatten(-1, (-1, group))
    return q.sub_(zero.float()[..., None]).mul_(step.float()[..., None]).flatten(-2)


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
    return x * (1 - 1 / (1 + torch.exp(2 * u)))     # x (1 + tanh u) / 2


def _adapter_term(st):
    """The adapters' term for every token, in fp32: X against all adapters, all but the token's own set to zero."""
    c = st["case"]
    L, R, T = c["L"], c["R"], c["T"]
    A, B = st["A"].float(), st["B"].float()
    ids = st["ids"].long()
    mine = (ids[:, None] == torch.arange(L, device=DEV)).float() * st["scale"]
    mask = mine[:, :, None]
    if st["ranks"] is not None:
        mask = mask * (torch.arange(R, device=DEV) < st["ranks"][:, None]).float()
    z = (st["X"].float() @ A.view(L * R, -1).T).view(T, L, R) * mask
    return z.view(T, L * R) @ B.transpose(1, 2).reshape(L * R, -1)


def _plain(st):
    c = st["case"]
    T = c["T"]
    if c["op"] == "route":
        x = st["logits"].float()
        order = torch.sort(x, dim=1, descending=True, stable=True)      # ties: the lowest index first
        top, ids = order.values[:, :c["topk"]], order.indices[:, :c["topk"]].to(torch.int32)
        if c["score"] == "softmax":
            big = torch.where(torch.isinf(order.values[:, :1]), 0.0, order.values[:, :1])
            w = torch.exp(top - big) / torch.exp(x - big).sum(1, keepdim=True).clamp(min=1e-30)
        else:
            w = 1 / (1 + torch.exp(-top))
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
        return [torch.where(torch.isinf(top), -1, ids), w]
    if c["op"] == "adapters":
        return (st["C"].float() + _adapter_term(st)).to(DTYPES[c["yt"]])
    bits, group = c["bits"], c["group"]
    if c["op"] == "shared":
        q = st["state"]
        y = (st["X"].float() / q["s"]) @ _weights(q["codes"], q["scale_f16"], q["zero_f16"], bits, group).T
        return (y + _adapter_term(st)).to(DTYPES[c["yt"]])
    E, I, k = c["E"], c["I"], c["topk"]
    gu, dn, ids = st["gate_up"], st["down"], st["ids"].long()
    x = st["X"].float() / gu["s"]
    if T * k < E:       # few pairs: the weights of each pair's expert
        at = ids.reshape(-1).clamp(min=0)
        wt = torch.where(ids < 0, 0.0, st["w"]).reshape(-1, 1)
        gate_up = _weights(gu["codes"][at], gu["scale_f16"][at], gu["zero_f16"][at], bits, group)
        h = torch.matmul(gate_up, x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        h = _act(h[:, :I], c["act"]) * h[:, I:] / dn["s"][at]
        down = _weights(dn["codes"][at], dn["scale_f16"][at], dn["zero_f16"][at], bits, group)
        y = (torch.matmul(down, h[:, :, None])[..., 0] * wt).view(T, k, -1).sum(1)
        return y.to(DTYPES[c["yt"]])
    # every expert for every token, weighted by the token's share of it
    share = torch.zeros((T, E), device=DEV).scatter_add_(1, ids.clamp(min=0), torch.where(ids < 0, 0.0, st["w"]))
    gate_up = _weights(gu["codes"], gu["scale_f16"], gu["zero_f16"], bits, group)
    h = (x @ gate_up.view(E * 2 * I, -1).T).view(T, E, 2 * I).transpose(0, 1)
    h = _act(h[:, :, :I], c["act"]) * h[:, :, I:] / dn["s"][:, None, :] * share.T[:, :, None]
    down = _weights(dn["codes"], dn["scale_f16"], dn["zero_f16"], bits, group)
    return torch.matmul(h, down.transpose(1, 2).contiguous()).sum(0).to(DTYPES[c["yt"]])


# ------------------------------------------------------------------ the definitions in 64 bits

def _w64(q, bits, group, e=None):
    """One matrix's (code - zero) step / s in fp64, its codes read bit by bit."""
    words, step, zero = (q[k] if e is None else q[k][e] for k in ("codes", "scale_f16", "zero_f16"))
    s = q["s"] if e is None or q["s"].dim() == 1 else q["s"][e]
    rows, cols = words.shape[0], words.shape[1] * 32 // bits
    v = torch.zeros((rows, cols), dtype=torch.float64, device=DEV)
    for b in range(bits):
        at = torch.arange(cols, device=DEV) * bits + b
        v += (((words[:, at >> 5] >> (at & 31).int()) & 1) << b).double()
    v = v.view(rows, cols // group, group)
    v.sub_(zero.double()[..., None]).mul_(step.double()[..., None])
    return v.view(rows, cols).div_(s.double())


def _gate64(x, act):
    if act == "silu":
        return x * torch.special.expit(x)
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    T = c["T"]
    if c["op"] == "route":
        x = st["logits"].double()
        order = torch.sort(x, dim=1, descending=True, stable=True)
        top = order.values[:, :c["topk"]]
        gone = top == -math.inf
        w = torch.softmax(x, 1).gather(1, order.indices[:, :c["topk"]]) if c["score"] == "softmax" else torch.special.expit(top)
        w = torch.where(gone, 0.0, w)
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, 0.0)
        return [torch.where(gone, -1, order.indices[:, :c["topk"]]).to(torch.int32), w]
    x = st["X"].double()
    if c["op"] == "moe":
        y = torch.zeros((T, c["K"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
            if t.numel() == 0:
                continue
            h = x[t] @ _w64(st["gate_up"], c["bits"], c["group"], e).T
            h = _gate64(h[:, :c["I"]], c["act"]) * h[:, c["I"]:]
            y.index_add_(0, t, (h @ _w64(st["down"], c["bits"], c["group"], e).T) * st["w"].double()[t, j][:, None])
        return y
    y = st["C"].double() if c["op"] == "adapters" else x @ _w64(st["state"], c["bits"], c["group"]).T
    for a in range(c["L"]):
        t = torch.nonzero(st["ids"] == a)[:, 0]
        if t.numel():
            r = c["R"] if st["ranks"] is None else int(st["ranks"][a])
            y[t] += (x[t] @ st["A"][a, :r].double().T) @ st["B"][a, :, :r].double().T * float(st["scale"][a])
    return y


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "route":
        return {"bytes": T * c["E"] * (4 if c["lt"] == "f32" else 2) + T * c["topk"] * 8, "flops": T * c["E"] * 4}
    xb, yb = (4 if c[k] == "f32" else 2 for k in ("xt", "yt"))
    per = (lambda: c["bits"] / 8 + 4 / c["group"])
    if c["op"] == "moe":
        pairs = T * c["topk"] * (0.75 if c["drop"] else 1)
        experts = c["E"] * (1 - (1 - 1 / c["E"]) ** pairs)          # distinct ones, as many as are expected
        if not c["drop"]:
            experts = max(experts, c["topk"])
        return {"bytes": experts * 3 * c["K"] * c["I"] * per() + T * c["K"] * (xb + yb) + T * c["topk"] * 8,
                "flops": 2 * pairs * 3 * c["K"] * c["I"]}
    ab = 4 if c["at"] == "f32" else 2
    have = T * (0.875 if c["none"] else 1)
    rank = (c["R"] + 1) / 2 if c["ragged"] else c["R"]
    adapters = min(c["L"], c["segments"] or have)
    n = {"bytes": adapters * rank * (c["K"] + c["M"]) * ab + T * (c["K"] * xb + c["M"] * yb), "flops": 2 * have * rank * (c["K"] + c["M"])}
    if c["op"] == "adapters":
        n["bytes"] += T * c["M"] * yb
    else:
        n["bytes"] += c["M"] * c["K"] * per() + 4 * c["K"]
        n["flops"] += 2 * T * c["M"] * c["K"]
    return n
