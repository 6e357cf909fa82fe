"""8-bit products by every kernel and in parts of the channels: an odd number of
128-channel steps, ragged ends, every kind of result; sums are exact, so results
equal their definition, or a call of few rows, whose kernel is another."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def codes_like(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def inputs(Tn, K, M, dt):
    g = torch.Generator(device="cuda").manual_seed(Tn + K + M)
    x, w = codes_like(g, Tn, K), codes_like(g, M, K)
    xs, ws = torch.rand(Tn, generator=g, device="cuda") + 0.5, torch.rand(M, generator=g, device="cuda") + 0.5
    sums = x.double() @ w.double().t().contiguous()      # whole numbers below 2^53
    return x, xs, w, ws, (sums.float() * xs[:, None] * ws[None, :]).to(DT[dt])


# Streamed for 32 rows at a time, in tiles of 64 x 32, 128 x 64, 256 x 128 and 256 x 256.
@pytest.mark.parametrize("Tn,K,M", [(17, 1840, 159), (139, 272, 65), (4193, 288, 332), (2429, 272, 2596), (3901, 288, 2624), (3901, 1328, 2624)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tiles_of_an_odd_number_of_steps(T, Tn, K, M, dt):
    say(f"gemm_i8 odd steps T={Tn} K={K} M={M} {dt}")
    assert -(-K // 128) % 2
    x, xs, w, ws, want = inputs(Tn, K, M, dt)
    for _ in range(2):
        assert torch.equal(T.ttq_gemm_i8(x, xs, w, ws, y_dtype=DT[dt]), want)


# The tiles, with 2 to 16 parts.
PARTS = [(145, 1888, 61), (131, 4976, 60), (2335, 4912, 269), (1421, 4432, 161), (797, 7472, 73), (433, 4976, 4728), (2085, 7792, 132), (3299, 9568, 542)]


@pytest.mark.parametrize("Tn,K,M", PARTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_parts(T, Tn, K, M, dt):
    """In parts, through a workspace of exactly the stated bytes between guards,
    full of NaN."""
    say(f"gemm_i8 parts T={Tn} K={K} M={M} {dt}")
    n = T.ttq_gemm_i8_workspace_bytes(Tn, K, M)
    assert n >= 2 * Tn * M * 4                           # the sums of two parts at least
    x, xs, w, ws, want = inputs(Tn, K, M, dt)
    big = torch.full((n + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(T.ttq_gemm_i8(x, xs, w, ws, y_dtype=DT[dt], ws=big[4096:4096 + n]), want)
    assert bool((big[:4096] == 0xFF).all()) and bool((big[4096 + n:] == 0xFF).all())


# Gate and up, and down, in tiles of 128 x 64, 256 x 128 and 256 x 256, with 1 to 23 steps.
@pytest.mark.parametrize("Tn,E,topk,K,I,M", [(109, 5, 2, 272, 2864, 68), (4225, 4, 2, 128, 336, 60), (5291, 3, 2, 128, 592, 61), (409, 5, 2, 128, 64, 2957),
                                             (1334, 2, 2, 128, 64, 2336), (2217, 3, 2, 128, 64, 2961), (1203, 3, 2, 272, 1408, 2063),
                                             (2000, 3, 2, 288, 1408, 2061), (700, 3, 2, 272, 1408, 1031)])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_layers_of_an_odd_number_of_steps(T, Tn, E, topk, K, I, M, yt):
    say(f"moe_i8 odd steps T={Tn} E={E} K={K} I={I} M={M} {yt}")
    g = torch.Generator(device="cuda").manual_seed(Tn + I)
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    X = torch.randn((Tn, K), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, E, (Tn, topk), generator=g, device="cuda", dtype=torch.int32)
    w = rand(Tn, topk) + 0.1
    up = dict(s=rand(K) + 0.5, codes=codes_like(g, E, 2 * I, K), scale=(rand(E, 2 * I) + 0.5) * (0.02 / K ** 0.5))
    down = dict(s=rand(E, I) + 0.5, codes=codes_like(g, E, M, I), scale=(rand(E, M) + 0.5) * (0.02 / I ** 0.5))
    every = T.ttq_moe_i8(X, ids, w, up, down, y_dtype=DT[yt])
    some = torch.cat([T.ttq_moe_i8(X[i:i + 64], ids[i:i + 64].contiguous(), w[i:i + 64].contiguous(), up, down, y_dtype=DT[yt])
                      for i in range(0, Tn, 64)])
    assert torch.isfinite(every).all() and torch.equal(every, some)


def test_two_captured_graphs_in_parts(T):
    """Two products in parts, each with its own workspace, captured and replayed
    in turn and at once, with eager work between."""
    say("two captured graphs, parts")
    jobs = []
    for Tn, K, M in ((145, 1888, 61), (1421, 4432, 161)):
        ws = torch.full((T.ttq_gemm_i8_workspace_bytes(Tn, K, M),), 0xFF, dtype=torch.uint8, device="cuda")
        assert ws.numel() >= 2 * Tn * M * 4
        x, xs, w, wsc, want = inputs(Tn, K, M, "f32")
        Y = torch.empty_like(want)
        jobs.append((lambda a=(x, xs, w, wsc), Y=Y, ws=ws: T.ttq_gemm_i8(*a, Y=Y, ws=ws), Y, want))
    graphs = []
    for run, _, _ in jobs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run()
        graphs.append((g, side))
    for turn in range(4):
        for _, Y, _ in jobs:
            Y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, side in graphs:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for run, Y, want in jobs:
            assert torch.equal(Y, want), turn
        jobs[turn % 2][0]()
        torch.cuda.synchronize()


@pytest.mark.parametrize("K,M", [(1040, 4097), (144, 6161), (4096, 40)])
def test_one_token_of_fp32_into_bf16(T, K, M):
    """One launch; equal to the same row in a call of two tokens."""
    say(f"qgemm_i8 one fp32 token K={K} M={M}")
    g = torch.Generator(device="cuda").manual_seed(K)
    X, s = torch.randn((2, K), generator=g, device="cuda"), torch.rand(K, generator=g, device="cuda") + 0.5
    W, ws = codes_like(g, M, K), torch.rand(M, generator=g, device="cuda")
    for sv in (s, None):
        one, two = (T.ttq_qgemm_i8(x, sv, W, ws, y_dtype=torch.bfloat16) for x in (X[:1], X))
        q, xs = T.ttq_quantize_rows(X, sv, divide=True)
        sums = q.double() @ W.double().t().contiguous()
        assert torch.equal(two, (sums.float() * xs[:, None] * ws[None, :]).bfloat16())
        assert torch.equal(one, two[:1])
