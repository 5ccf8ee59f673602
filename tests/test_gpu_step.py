"""A fine-tuning step of a whole layer: PactLayer with its attention core (rotation, packed causal
attention and their gradients) and its adapters' update, in the composition a user runs."""
import numpy as np
import pytest
import torch

import synth
from tests import ref64

pytestmark = pytest.mark.gpu

SMALL = dict(H=512, I=768, KV=256, batch=1, seq=300, outliers=False)


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def build(monkeypatch, D=64, M=300, starts=(0, 130, 130, 131, 290), attention=True, **kw):
    from nvfp4_gemm_b200.layer import AttentionCore, LayerShape, PactLayer
    monkeypatch.setitem(synth.LAYERS, "small", SMALL)
    inp = synth.layer_inputs("small", M=M)
    freq = [1e6 ** (-2 * i / D) for i in range(D // 2)]
    core = AttentionCore(D, torch.tensor(starts, dtype=torch.int32, device="cuda"), freq) if attention else None
    part = lambda key: {k: dev(v) for k, v in inp[key].items()}
    L = PactLayer(LayerShape(M=M, H=SMALL["H"], I=SMALL["I"], KV=SMALL["KV"]), part("w"), part("lora_a"),
                  part("lora_b"), dev(inp["gamma1"]), dev(inp["gamma2"]), attention=core, **kw)
    return L, inp, freq


@pytest.mark.parametrize("D", [64, 128])
def test_layer_with_attention_core(monkeypatch, D):
    """The core's stages against their 64-bit forms on the layer's own tensors, and everything else bit
    for bit against the layer that is given the same attn and d_qkv."""
    import nvfp4_gemm_b200 as P
    L, inp, freq = build(monkeypatch, D)
    h, d_out = dev(inp["h"]), dev(inp["d_out"])
    L.bind(h, d_out)
    L.step()
    torch.cuda.synchronize()
    assert P.pact_get_device_status() == 0, P.pact_last_error()
    S, n = L.s, 290
    given, _, _ = build(monkeypatch, D, attention=False)
    given.bind(h, L.attn, d_out, L.d_qkv)
    given.step()
    torch.cuda.synchronize()
    for name in ("out", "dh", "dattn"):
        assert torch.equal(getattr(L, name), getattr(given, name)), name
    for k in L.grads:
        assert torch.equal(L.grads[k], given.grads[k]), k
    # rotation: padding rows and v stay as the projection wrote them
    qk = slice(0, S.H + S.KV)
    assert torch.equal(L.qkv[:, S.H + S.KV:], given.qkv[:, S.H + S.KV:])
    assert torch.equal(L.qkv[n:], given.qkv[n:])
    place = torch.cat([torch.arange(130), torch.arange(1), torch.arange(159)]).cuda()
    assert torch.equal(L.pos[:n].long(), place) and bool((L.pos[n:] == -1).all())
    ref64.within(L.qkv[:n, qk], ref64.rope(given.qkv[:n, qk], place, freq, L.heads + L.kv_heads), "rotated q, k")
    q, k, v = L.qkv[:, :S.H], L.qkv[:, S.H:S.H + S.KV], L.qkv[:, S.H + S.KV:]
    ref = ref64.attention(q, k, v, [0, 130, 131, 290], L.heads, L.kv_heads, D ** -0.5, L.dattn, L.attn)
    ref64.within(L.attn, ref["o"], "attn")
    ref64.within(L.lse, ref["lse"], "lse")
    # d(qkv): the core's gradient, turned back by the rotation (its own rounding on top)
    for name, cols, heads in (("dq", slice(0, S.H), L.heads), ("dk", slice(S.H, S.H + S.KV), L.kv_heads)):
        value, bound = (t[:n] for t in ref[name])
        back, size = ref64.rope(value, place, freq, heads, inverse=True)
        # both members of a pair carry their bound into both members of the result
        pair = bound.reshape(n, heads, 2, D // 2).sum(2, keepdim=True).expand(-1, -1, 2, -1).reshape(n, -1)
        ref64.within(L.d_qkv[:n, cols], (back, 1.01 * (pair + size)), f"d {name}")
    ref64.within(L.d_qkv[:, S.H + S.KV:], ref["dv"], "dv")
    assert not L.attn[n:].any() and not L.d_qkv[n:].any()
    assert L.saved_bytes() == given.saved_bytes() + 2 * S.M * S.n_qkv + 4 * L.heads * S.M


def test_steps_with_updates_captured_and_eager(monkeypatch):
    """Three steps, each forward, backward and update: eager, and as one captured graph replayed with the
    LoRA gradients on a side stream, give the same adapters bit for bit."""
    runs = []
    for captured in (False, True):
        L, inp, _ = build(monkeypatch, trainable=True)
        L.bind(dev(inp["h"]), dev(inp["d_out"]))
        if captured:
            side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            L.step()    # first calls set per-device attributes
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                L.step_concurrent(side)
                L.update(lr=0.02, weight_decay=0.01)
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(3):
                L.step()
                L.update(lr=0.02, weight_decay=0.01)
        torch.cuda.synchronize()
        runs.append(L)
    a, b = runs
    for k in a.masters:
        assert torch.equal(a.masters[k], b.masters[k]) and torch.equal(a.momenta[k], b.momenta[k]), k
        assert torch.equal(a.adapters[k], a.masters[k].bfloat16()), k


def test_captured_step_follows_another_packing(monkeypatch):
    """pack() changes the sequences of a captured step; rows that became padding hold zeros."""
    L, inp, _ = build(monkeypatch)
    L.bind(dev(inp["h"]), dev(inp["d_out"]))
    L.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step()
    graph.replay()
    other = (0, 40, 200, 200, 220)
    L.pack(torch.tensor(other, dtype=torch.int32, device="cuda"))
    graph.replay()
    fresh, _, _ = build(monkeypatch, starts=other)
    fresh.bind(dev(inp["h"]), dev(inp["d_out"]))
    fresh.step()
    torch.cuda.synchronize()
    for name in ("attn", "lse", "d_qkv", "out", "dh"):
        assert torch.equal(getattr(L, name), getattr(fresh, name)), name
    assert not L.attn[220:].any() and not L.d_qkv[220:].any()


@pytest.mark.parametrize("fp32", [False, True])
def test_update_matches_the_64_bit_form(monkeypatch, fp32):
    """The 14 matrices of the stacked adapters, from the layer's own gradients."""
    L, inp, _ = build(monkeypatch, trainable=True, grad_fp32=fp32)
    given = {k: t.clone() for k, t in L.adapters.items()}
    assert all(t.data_ptr() != dev_t.data_ptr() for t, dev_t in zip(L.adapters.values(), given.values()))
    L.bind(dev(inp["h"]), dev(inp["d_out"]))
    L.step()
    grads = L._matrices(L.grads32 if fp32 else L.grads)
    assert len(grads) == 14
    w, m = [t.clone() for t in L._matrices(L.masters)], [t.clone() for t in L._matrices(L.momenta)]
    L.update(lr=0.05, momentum=0.9, weight_decay=0.1)
    torch.cuda.synchronize()
    for i, (w1, m1) in enumerate(zip(L._matrices(L.masters), L._matrices(L.momenta))):
        pm, pw = ref64.muon(w[i], grads[i], m[i], 0.05, 0.9, 0.1)
        ref64.within(m1, pm, f"momentum {i}")
        ref64.within(w1, pw, f"weight {i}")


def test_update_needs_a_trainable_layer(monkeypatch):
    L, inp, _ = build(monkeypatch)
    with pytest.raises(RuntimeError):
        L.update(lr=0.1)
    for args, kw in (((1,), {}), ((1, 2, 3), {}), ((1,), {"h": 2}), ((1,), {"attn": 2})):
        with pytest.raises(TypeError):
            L.bind(*args, **kw)
    L.bind(d_out=2, h=1)
    assert L.inputs == (1, L.attn, 2, L.d_qkv)


def test_workspaces_off_the_device_are_refused():
    import nvfp4_gemm_b200 as P
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    o, lse = P.pact_attention_fwd(x, x, x, cu, 2, 2)
    w = [torch.zeros((4, 8), device="cuda")]
    big = torch.zeros((1 << 16, 2), dtype=torch.uint8)
    for ws, error in ((big, TypeError), (big.cuda()[:, 0], ValueError)):
        with pytest.raises(error):
            P.pact_attention_bwd(x, x, x, x, o, lse, cu, 2, 2, workspace=ws)
        with pytest.raises(error):
            P.pact_muon_step(w, w, w, lr=0.1, weights_out=[w[0].clone()], momenta_out=[w[0].clone()], workspace=ws)
    assert not w[0].any()


def test_angles_on_the_device_are_captured_too(monkeypatch):
    """inv_freq as a device tensor: read once, so that a captured step needs no copy of it."""
    from nvfp4_gemm_b200.layer import AttentionCore
    want, inp, freq = build(monkeypatch)
    monkeypatch.setattr("nvfp4_gemm_b200.layer.AttentionCore", lambda D, starts, f: AttentionCore(
        D, starts, torch.tensor(f, dtype=torch.float64, device="cuda")))
    got, _, _ = build(monkeypatch)
    for L in (want, got):
        L.bind(dev(inp["h"]), dev(inp["d_out"]))
        L.step()
    torch.cuda.synchronize()
    for t in (got.qkv, got.out, got.dh):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.step()
    graph.replay()
    torch.cuda.synchronize()
    for name in ("qkv", "out", "dh"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name


def test_an_updated_layer_is_the_layer_of_the_new_adapters(monkeypatch):
    """Nothing a layer keeps goes back to the adapters it was built with."""
    from nvfp4_gemm_b200.layer import PactLayer
    L, inp, _ = build(monkeypatch, trainable=True)
    L.bind(dev(inp["h"]), dev(inp["d_out"]))
    L.step()
    L.update(lr=0.5)
    before = L.out.clone()
    L.step()
    a_q, a_k, a_v, b_q, b_k, b_v, a_o, b_o, a_g, a_u, b_g, b_u, a_d, b_d = [t.clone() for t in L._matrices(L.adapters)]
    fresh = PactLayer(L.s, {k: dev(v) for k, v in inp["w"].items()},
                      {"q": a_q, "k": a_k, "v": a_v, "o": a_o, "gate": a_g, "up": a_u, "down": a_d},
                      {"q": b_q, "k": b_k, "v": b_v, "o": b_o, "gate": b_g, "up": b_u, "down": b_d},
                      dev(inp["gamma1"]), dev(inp["gamma2"]), attention=L.attention)
    fresh.bind(dev(inp["h"]), dev(inp["d_out"]))
    fresh.step()
    torch.cuda.synchronize()
    assert not torch.equal(before, L.out)
    for name in ("out", "dh", "d_qkv"):
        assert torch.equal(getattr(L, name), getattr(fresh, name)), name
    for k in L.grads:
        assert torch.equal(L.grads[k], fresh.grads[k]), k


@pytest.mark.parametrize("raw", [False, True])
def test_memory_for_another_stream_is_not_the_current_streams(raw):
    """A call on another stream takes neither its outputs nor its scratch from a block that was just freed on
    the current stream while work is pending there."""
    import nvfp4_gemm_b200 as P
    M, hq, hk, D = 512, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = lambda n: torch.randn((M, n), generator=g, device="cuda").bfloat16()
    q, k, v, do = bf(hq * D), bf(hk * D), bf(hk * D), bf(hq * D)
    cu = torch.tensor([0, 200, M], dtype=torch.int32, device="cuda")
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    freq = [1e4 ** (-2 * i / D) for i in range(D // 2)]
    w, grad = torch.randn((64, 3000), generator=g, device="cuda"), torch.randn((64, 3000), generator=g, device="cuda")

    def calls(stream):
        o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk, stream=stream)
        w1, m1 = w.clone(), torch.zeros_like(w)
        torch.cuda.current_stream().synchronize()      # the copies, before the other stream updates them
        return [lambda: [P.pact_rope(q, pos, freq, hq, stream=stream)],
                lambda: list(P.pact_attention_fwd(q, k, v, cu, hq, hk, stream=stream)),
                lambda: list(P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk, stream=stream)),
                lambda: [P.pact_muon_step([w1], [grad], [m1], lr=0.1, stream=stream), w1, m1][1:]]
    want = [f() for f in calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    todo = calls(side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    sizes = [M * hq * D * 2, M * hk * D * 2, M * hq * 4, P.pact_attention_bwd_workspace_bytes(M, hq),
             P.pact_muon_workspace_bytes([w.shape])]
    for f, ref in zip(todo, want):
        blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        kept = [torch.empty_like(b) for b in blocks]
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)       # some 25 ms of the current stream, ahead of its reads of the blocks
        for a, b in zip(kept, blocks):
            a.copy_(b)
        begin = {b.data_ptr() for b in blocks}
        del blocks, b
        got = f()
        side.synchronize()
        assert not begin & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(bool((a == 7).all()) for a in kept)
