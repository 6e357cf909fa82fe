"""8-bit layers and sorted rows: streams, captured graphs, workspaces, and
addresses that pass 32 bits."""
import numpy as np
import pytest
import torch

import i8_ref as ref
from gpu_util import f32_dev, host, i32_dev, say
from test_gpu_i8 import enc, i8_dev, moe_inputs, moe_ref, near, rounded, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def layer(T, seed, Tn, E, topk, K, I, M):
    d = moe_inputs(seed, Tn, E, topk, K, I, M, "bf16", False, True, True)
    ws = torch.full((T.ttq_moe_i8_workspace_bytes(Tn, topk, K, I, M, E),), 0xFF, dtype=torch.uint8, device="cuda")
    ids, w = i32_dev(d["ids"]), f32_dev(d["w"])
    Y = torch.empty((Tn, M), dtype=torch.bfloat16, device="cuda")

    def run():
        T.ttq_moe_i8(d["X"], ids, w, d["gate_up"], d["down"], Y=Y, ws=ws)
    return run, Y, d


def product(T, seed, Tn, K, M):
    """A projection; few tiles and many channels: in parts, through the workspace."""
    rng = np.random.default_rng(seed)
    X, x = enc(rng.standard_normal((Tn, K)), "bf16")
    wq, ws = rng.integers(-127, 128, (M, K)).astype(np.int8), rng.random(M).astype(np.float32)
    W, wsd = i8_dev(wq), f32_dev(ws)
    scratch = torch.full((T.ttq_qgemm_i8_workspace_bytes(Tn, K, M),), 0xFF, dtype=torch.uint8, device="cuda")
    Y = torch.empty((Tn, M), device="cuda")

    def run():
        T.ttq_qgemm_i8(X, None, W, wsd, Y=Y, ws=scratch)
    return run, Y, ref.product(*ref.quantize(x), wq, ws)


def test_two_captured_graphs(T):
    """Graphs of a layer and of projections, each with its own workspace,
    replayed in turn and at once, with eager work between."""
    say("two captured graphs")
    jobs = [layer(T, 3, 70, 6, 2, 256, 192, 130), layer(T, 4, 2, 6, 2, 256, 192, 130), product(T, 5, 1, 4096, 300), product(T, 6, 40, 8192, 200)]
    graphs, eager = [], []
    for run, Y, _ in jobs:
        run()
        eager.append(Y.clone())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run()
        graphs.append(g)
    same(eager[2], jobs[2][2])
    same(eager[3], jobs[3][2])
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(4):
        for _, Y, _ in jobs:
            Y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, Y, _), e in zip(jobs, eager):
            assert torch.equal(Y, e), turn
        jobs[turn][0]()                                   # eager work between replays
        torch.cuda.synchronize()


def test_streams(T):
    """On a stream that is not the current one, by torch stream and by handle;
    what the call allocates belongs to it."""
    say("streams")
    rng = np.random.default_rng(8)
    x = rng.standard_normal((50, 512)).astype(np.float32)
    wq, ws = ref.quantize(rng.standard_normal((200, 512)))
    X, W, wsd = f32_dev(x), i8_dev(wq), f32_dev(ws)
    want = ref.product(*ref.quantize(x), wq, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        Y = T.ttq_qgemm_i8(X, None, W, wsd, stream=stream)
        s.synchronize()
        same(Y, want)
    pos = T.ttq_moe_sort(i32_dev(rng.integers(0, 4, (50, 2))), 4, stream=s)[2]
    R = T.ttq_moe_gather(X, pos, stream=s)
    Y = T.ttq_moe_combine(R, pos, stream=s)
    s.synchronize()
    assert torch.equal(Y, 2 * X)


@pytest.mark.parametrize("Tn,K,M", [(40, 8192, 200), (17, 14336, 70), (200, 4096, 1000), (100, 8192, 33)])
def test_parts_with_a_workspace_of_the_stated_size(T, Tn, K, M):
    """A workspace of exactly the stated bytes between guards: nothing is
    written around it."""
    say(f"workspace guards T={Tn} K={K} M={M}")
    rng = np.random.default_rng(K)
    xq, wq = rng.integers(-127, 128, (Tn, K)), rng.integers(-127, 128, (M, K))
    xs, ws = rng.random(Tn).astype(np.float32), rng.random(M).astype(np.float32)
    n = T.ttq_gemm_i8_workspace_bytes(Tn, K, M)
    big = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    Y = T.ttq_gemm_i8(i8_dev(xq), f32_dev(xs), i8_dev(wq), f32_dev(ws), ws=big[4096:4096 + n])
    same(Y, ref.product(xq, xs, wq, ws))
    assert bool((big[:4096] == 0xA5).all()) and bool((big[4096 + n:] == 0xA5).all())


def test_rows_beyond_32_bits(T):
    """Rows 2^22 codes apart, so that the last of X, W and R lie behind 2^32
    bytes of the first."""
    say("addresses beyond 32 bits")
    rng = np.random.default_rng(1)
    ld, n, K = 1 << 22, 1100, 160
    big = torch.zeros((n, ld), dtype=torch.int8, device="cuda")
    xq = rng.integers(-127, 128, (n, K)).astype(np.int8)
    big[:, :K] = i8_dev(xq)
    some = rng.integers(-127, 128, (70, K)).astype(np.int8)
    one, ws = np.ones(n, np.float32), rng.random(70).astype(np.float32)
    same(T.ttq_gemm_i8(big[:, :K], f32_dev(one), i8_dev(some), f32_dev(ws)), ref.product(xq, one, some, ws))
    same(T.ttq_gemm_i8(i8_dev(some), f32_dev(ws), big[:, :K], f32_dev(one)), ref.product(some, ws, xq, one))
    few = some[:3]
    same(T.ttq_gemm_i8(i8_dev(few), f32_dev(ws[:3]), big[:, :K], f32_dev(one)), ref.product(few, ws[:3], xq, one))
    # rows of fp32, 2^20 apart: read and written by the row calls
    wide = big.view(torch.float32)[:, :K]
    x = rng.standard_normal((n, K)).astype(np.float32)
    wide.copy_(f32_dev(x))
    q, sc = T.ttq_quantize_rows(wide)
    rq, rs = ref.quantize(x)
    same(sc, rs)
    np.testing.assert_array_equal(host(q), rq)
    pos = i32_dev(rng.permutation(n).reshape(n, 1))
    Y = T.ttq_moe_combine(wide, pos)
    assert torch.equal(Y, f32_dev(x)[pos[:, 0].long()])
    dR, dw = T.ttq_moe_combine_grad(Y, wide, pos)
    assert torch.equal(dR, f32_dev(x))
    out = T.ttq_moe_gather(Y, pos, R=wide)
    assert torch.equal(out, f32_dev(x))


def test_the_same_expert_twice_and_ids_beyond(T):
    """A token that names an expert twice counts it twice; ids of other places
    add nothing and their weights are not read."""
    say("moe_i8 twice")
    d = moe_inputs(21, 9, 4, 2, 64, 48, 20, "f32", False, False, False)
    ids, w = d["ids"], d["w"].copy()
    ids[:, 1] = ids[:, 0]
    twice = T.ttq_moe_i8(d["X"], i32_dev(ids), f32_dev(w), d["gate_up"], d["down"])
    once = ids.copy()
    once[:, 1] = 4
    sums = w.copy()
    sums[:, 0] = w[:, 0] + w[:, 1]
    sums[:, 1] = np.nan
    single = T.ttq_moe_i8(d["X"], i32_dev(once), f32_dev(sums), d["gate_up"], d["down"])
    # w0 v + w1 v in two roundings against (w0 + w1) v: both terms positive multiples of v
    assert torch.all((twice - single).abs() <= 4 * 2.0 ** -24 * single.abs())


def test_quantized_state_and_projection_of_a_prompt(T):
    """Statistics, scales, an 8-bit weight and the projection: the run of a
    prompt, against the same steps in fp64."""
    say("prompt in 8 bits")
    rng = np.random.default_rng(4)
    X, x = enc(rng.standard_normal((130, 768)) * np.where(rng.random(768) < 0.02, 20, 1), "bf16")
    w = rng.standard_normal((300, 768)).astype(np.float32) * 0.02
    ssq = T.ttq_stats(X, torch.empty(768, dtype=torch.float64, device="cuda"))
    s = T.ttq_awq_scales(ssq, 130, 0.5, 0.01)
    W, ws = T.ttq_quantize_rows(f32_dev(w), s)
    Y = T.ttq_qgemm_i8(X, s, W, ws)
    sh = host(s)
    same(Y, ref.product(*ref.quantize(x, sh, True), *ref.quantize(w, sh)))
    # and a shared input, quantized once for two projections
    q, xs = T.ttq_quantize_rows(X, s, divide=True)
    assert torch.equal(T.ttq_gemm_i8(q, xs, W, ws), Y)
    assert torch.equal(T.ttq_gemm_i8(q, xs, W[100:200], ws[100:200]), Y[:, 100:200])
    same(T.ttq_gemm_i8(q, xs, W, ws, y_dtype=torch.bfloat16), rounded(host(Y), "bf16"))


@pytest.mark.parametrize("Tn,topk,K,per_in", [(600, 1, 64, False), (1024, 2, 32, False), (1025, 2, 32, False), (3, 2, 16400, False),
                                              (5, 3, 16384, False), (600, 3, 32, True)])
def test_moe_sorted_beside_the_rows(T, Tn, topk, K, per_in):
    """Few slots are sorted while the tokens' rows are quantized: more rows than
    workgroups, the most slots of it and one token more, channels that a workgroup
    holds and that it does not."""
    say(f"moe_i8 sorted beside the rows T={Tn} topk={topk} K={K}")
    d = moe_inputs(Tn + K, Tn, 3, topk, K, 48, 20, "bf16", per_in, False, True)
    ws = torch.full((T.ttq_moe_i8_workspace_bytes(Tn, topk, K, 48, 20, 3),), 0xFF, dtype=torch.uint8, device="cuda")
    Y = T.ttq_moe_i8(d["X"], i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"], ws=ws)
    near(Y, *moe_ref(d, "silu"), "f32")


def codes_like(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("Tn,K,M", [(2048, 528, 4100), (2001, 1040, 4000), (2300, 1072, 4097), (1024, 14336, 2050), (40, 8208, 1030)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gemm_of_many_tiles(T, Tn, K, M, dt):
    """The largest tiles, with ragged ends, and channels in parts: the exact
    sums in fp64, the scales in fp32."""
    say(f"gemm_i8 many tiles T={Tn} K={K} M={M} {dt}")
    g = torch.Generator(device="cuda").manual_seed(Tn + K + M)
    x, w = codes_like(g, Tn, K), codes_like(g, M, K)
    xs, ws = torch.rand(Tn, generator=g, device="cuda"), torch.rand(M, generator=g, device="cuda")
    sums = x.double() @ w.double().t().contiguous()      # whole numbers below 2^53
    want = (sums.float() * xs[:, None] * ws[None, :]).to(dt)
    for turn in range(2):
        assert torch.equal(T.ttq_gemm_i8(x, xs, w, ws, y_dtype=dt), want)


@pytest.mark.parametrize("Tn,K,I,M,E,topk", [(1500, 2064, 2000, 1030, 2, 2), (4000, 1056, 1040, 1056, 2, 2), (4003, 1056, 1040, 1054, 5, 2),
                                             (4000, 528, 2000, 1056, 3, 1)])
def test_moe_of_many_tiles(T, Tn, K, I, M, E, topk):
    """The largest tiles give every token what a call of a few tokens gives it,
    whose tiles are others."""
    say(f"moe_i8 many tiles T={Tn} K={K} I={I} M={M} E={E}")
    g = torch.Generator(device="cuda").manual_seed(Tn + I)
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    X = torch.randn((Tn, K), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, E, (Tn, topk), generator=g, device="cuda", dtype=torch.int32)
    w = rand(Tn, topk)
    up = dict(s=rand(K) + 0.5, codes=codes_like(g, E, 2 * I, K), scale=rand(E, 2 * I) * (0.02 / K ** 0.5))
    down = dict(s=rand(E, I) + 0.5, codes=codes_like(g, E, M, I), scale=rand(E, M) * (0.02 / I ** 0.5))
    every = T.ttq_moe_i8(X, ids, w, up, down)
    assert torch.isfinite(every).all()
    for lo, n in ((0, 100), (Tn // 2, 37), (Tn - 64, 64), (Tn - 1, 1)):
        part = T.ttq_moe_i8(X[lo:lo + n], ids[lo:lo + n].contiguous(), w[lo:lo + n].contiguous(), up, down)
        assert torch.equal(part, every[lo:lo + n]), lo
