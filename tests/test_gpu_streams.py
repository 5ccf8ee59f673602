"""Calls given a stream of their own: what they allocate is that stream's memory, not a block that the
current stream may still be using, and the results are those of the current stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu

M, K, N, r = 256, 512, 384, 16


def tensors(x):
    """The tensors of a call's results."""
    import nvfp4_gemm_b200 as P
    if isinstance(x, torch.Tensor):
        return [x]
    if isinstance(x, P.NVFP4Tensor):
        return [x.codes, x.scales]
    if isinstance(x, P.WeightCache):
        return [x.buf]
    return [t for y in x for t in tensors(y)] if isinstance(x, (list, tuple)) else []


def calls():
    """(name, call of a stream), on inputs that are complete."""
    import nvfp4_gemm_b200 as P
    g = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *sh: torch.randn(sh, generator=g, device="cuda").bfloat16()
    x, dy, W, A, B = bf(M, K), bf(M, N), bf(N, K) * 0.02, bf(r, K) * 0.02, bf(N, r) * 0.02
    gamma, gate, up = bf(K), bf(M, K), bf(M, K)
    wc, xq, dyq = P.pact_weight_layout_cache(W), P.pact_quantize_nvfp4(x), P.pact_quantize_nvfp4(dy)
    T, U = P.pact_lora_fwd(x, A, 2.0), P.pact_lora_bwd_u(dy, B, r, [N], 2.0)
    yq, _, rstd = P.pact_rmsnorm_quant(x, gamma, 1e-5)
    _, _, gq, uq = P.pact_silu_mul_quant(gate, up)
    lf, lb = P.lora_struct(T, B, r, [N]), P.lora_struct(U, A, r, [K])
    wf = wc.fwd
    torch.cuda.synchronize()
    return [
        ("quantize", lambda s: P.pact_quantize_nvfp4(x, stream=s)),
        ("rmsnorm_quant", lambda s: P.pact_rmsnorm_quant(x, gamma, 1e-5, stream=s)),
        ("silu_mul_quant", lambda s: P.pact_silu_mul_quant(gate, up, stream=s)),
        ("absmax", lambda s: P.pact_absmax_bf16(W, stream=s)),
        ("layout_cache", lambda s: P.pact_weight_layout_cache(W, stream=s)),
        ("layout_cache_two_level", lambda s: P.pact_weight_layout_cache(W, stream=s, two_level=True)),
        ("layout_cache_from_nvfp4", lambda s: P.pact_weight_layout_cache_from_nvfp4(wf, stream=s)),
        ("gptq", lambda s: P.pact_gptq_nvfp4(W, x, stream=s)),
        ("gemm_fwd", lambda s: P.pact_frozen_gemm_fwd(xq, wc, lf, stream=s)),
        ("gemm_dgrad", lambda s: P.pact_frozen_gemm_dgrad(dyq, wc, lb, stream=s)),
        ("lora_fwd", lambda s: P.pact_lora_fwd(x, A, 2.0, stream=s)),
        ("lora_fwd_noalloc", lambda s: P.pact_lora_fwd_noalloc(x, A, 2.0, stream=s)),
        ("lora_bwd_u", lambda s: P.pact_lora_bwd_u(dy, B, r, [N], 2.0, stream=s)),
        ("lora_bwd", lambda s: P.pact_lora_bwd(dy, A, U, r, [N], 2.0, x=x, stream=s)),
        ("round", lambda s: P.pact_round_bf16(rstd, stream=s)),
        ("silu_mul_bwd", lambda s: P.pact_silu_mul_bwd_quant(gate, gq, uq, want_m=True, stream=s)),
        ("rmsnorm_bwd", lambda s: P.pact_rmsnorm_bwd(x, yq, rstd, gamma, want_q=True, stream=s)),
    ]


def test_memory_of_the_calls_stream():
    """Blocks of each result's size, just freed on the current stream with work pending that reads them, are
    neither handed out nor written."""
    import nvfp4_gemm_b200 as P
    todo = calls()
    want = [tensors(f(None)) for _, f in todo]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for (name, f), ref in zip(todo, want):
        blocks = [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device="cuda") for t in ref]
        kept = [torch.empty_like(b) for b in blocks]
        torch.cuda.synchronize()
        torch.cuda._sleep(5_000_000)       # a few ms of the current stream, ahead of its reads of the blocks
        for a, b in zip(kept, blocks):
            a.copy_(b)
        begin = {b.data_ptr() for b in blocks}
        del blocks, b
        got = tensors(f(side))
        side.synchronize()
        assert not begin & {t.data_ptr() for t in got}, name
        torch.cuda.synchronize()
        assert all(bool((a == 7).all()) for a in kept), name
        assert len(got) == len(ref), name
        # (a cache's padding between its parts is never written)
        if "layout_cache" not in name:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref)), name
    assert P.pact_get_device_status() == 0, P.pact_last_error()


def test_captured_on_a_second_stream():
    """A fork of a captured step that gives its calls the second stream: their memory is the graph's."""
    import nvfp4_gemm_b200 as P
    g = torch.Generator(device="cuda").manual_seed(4)
    hq, hk, D = 4, 2, 64
    bf = lambda n: torch.randn((300, n), generator=g, device="cuda").bfloat16()
    q, k, v, do = bf(hq * D), bf(hk * D), bf(hk * D), bf(hq * D)
    cu = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")

    def step(stream):
        o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk, stream=stream)
        grads = P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk, stream=stream)
        return [o, lse, *grads, *tensors(P.pact_quantize_nvfp4(grads[0], stream=stream))]
    want = step(None)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        other = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(4)]   # work beside the graph's memory
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(got, want, copies))
    assert all(bool((t == 3.0).all()) for t in other)
