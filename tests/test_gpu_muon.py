"""pact_muon_step against the Newton-Schulz products in 64 bits: both orientations, ranks, odd
lengths and alignments, batches, gradients of both types, zero and near low-rank gradients."""
import pytest
import torch

from tests import ref64

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 9), (5, 1), (16, 16), (16, 2048), (2048, 16), (16, 1023), (1025, 16), (17, 300), (300, 31),
          (32, 513), (48, 260), (257, 48), (64, 64), (64, 1000), (999, 64), (3, 70000)]


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def step_and_check(w, g, m, nesterov=True, wd=0.01, out=None):
    import nvfp4_gemm_b200 as P
    n = len(w)
    ref = [ref64.muon(w[i], g[i], m[i], 0.02, 0.95, wd, nesterov) for i in range(n)]
    w16 = [torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in w]
    mo, wo = (None, None) if out is None else out
    P.pact_muon_step(w, g, m, lr=0.02, momentum=0.95, weight_decay=wd, nesterov=nesterov, weights_out=wo,
                     momenta_out=mo, weights_bf16=w16)
    torch.cuda.synchronize()
    for i in range(n):
        ref64.within((mo or m)[i], ref[i][0], f"m {tuple(w[i].shape)}")
        ref64.within((wo or w)[i], ref[i][1], f"W {tuple(w[i].shape)}")
        assert torch.equal(w16[i], (wo or w)[i].bfloat16())


@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_one_matrix(shape, gdt):
    step_and_check([rnd(1, *shape, std=0.02)], [rnd(2, *shape, std=1e-3).to(gdt)], [rnd(3, *shape, std=1e-3)])


@pytest.mark.parametrize("nesterov", [True, False])
def test_many_matrices_of_all_shapes_out_of_place(guards, nesterov):
    """More matrices than one launch takes, in guarded buffers that start off 16-byte alignment."""
    shapes = (SHAPES * 9)[:150]

    def buffers(seed, std):
        out = []
        for i, (a, b) in enumerate(shapes):
            t = guards.flat(4 * a * b + 4 * (i % 2))[4 * (i % 2):].view(torch.float32).view(a, b)
            t.copy_(rnd(seed + i, a, b, std=std))
            out.append(t)
        return out
    w, g, m = buffers(0, 0.02), buffers(1000, 1e-3), buffers(2000, 1e-3)
    wo, mo = buffers(0, 0.0), buffers(0, 0.0)
    kept = [t.clone() for t in w + g + m]
    step_and_check(w, g, m, nesterov, out=(mo, wo))
    assert all(torch.equal(a, b) for a, b in zip(kept, w + g + m)), "an input changed"


def test_batched_tensors_match_single_matrices():
    import nvfp4_gemm_b200 as P
    w, g, m = rnd(1, 5, 16, 200), rnd(2, 5, 16, 200), rnd(3, 5, 16, 200)
    w2, m2 = w.clone(), m.clone()
    P.pact_muon_step([w], [g], [m], lr=0.1)
    for i in range(5):
        P.pact_muon_step([w2[i]], [g[i]], [m2[i]], lr=0.1)
    assert torch.equal(w, w2) and torch.equal(m, m2)


def test_zero_and_low_rank_gradients():
    a, b = rnd(1, 16, 1), rnd(2, 1, 3000)
    z = torch.zeros((16, 3000), device="cuda")
    w = [rnd(3, 16, 3000, std=0.02) for _ in range(3)]
    import nvfp4_gemm_b200 as P
    # no gradient and no momentum: the weight only decays
    w0 = w[0].clone()
    P.pact_muon_step([w0], [z], [z.clone()], lr=0.02, weight_decay=0.5)
    assert torch.equal(w0, (0.99 * w[0].double()).float())
    # one direction, and one direction with a faint rest
    step_and_check([w[1]], [a @ b], [z.clone()])
    step_and_check([w[2]], [a @ b + 1e-5 * rnd(5, 16, 3000)], [z.clone()])


def test_repeats_captures_and_streams():
    import nvfp4_gemm_b200 as P
    w, g, m = [rnd(1, 16, 5000), rnd(2, 700, 16)], [rnd(3, 16, 5000), rnd(4, 700, 16)], [rnd(5, 16, 5000), rnd(6, 700, 16)]
    outs = [[torch.empty_like(t) for t in w] for _ in range(4)]
    mo = [[torch.empty_like(t) for t in w] for _ in range(4)]
    P.pact_muon_step(w, g, m, lr=0.1, weights_out=outs[0], momenta_out=mo[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        P.pact_muon_step(w, g, m, lr=0.1, weights_out=outs[1], momenta_out=mo[1])
    side.synchronize()
    ws = torch.empty(P.pact_muon_workspace_bytes([t.shape for t in w]), dtype=torch.uint8, device="cuda")
    graphs = []
    for i in (2, 3):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            P.pact_muon_step(w, g, m, lr=0.1, weights_out=outs[i], momenta_out=mo[i], workspace=ws)
    for i in (0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in (1, 2, 3):
        assert all(torch.equal(x, y) for x, y in zip(outs[i] + mo[i], outs[0] + mo[0]))


def test_clusters_and_slabs_in_one_call():
    """Matrices that fit a cluster, alone and in batches, between ones that take the slabs of scratch, of
    more than one launch each."""
    shapes = [(16, 700), (2, 3, 70001), (300, 9), (3, 16, 520), (12, 60000), (1, 1)] * 22
    w = [rnd(i, *s, std=0.02) for i, s in enumerate(shapes)]
    g, m = [rnd(500 + i, *s, std=1e-3) for i, s in enumerate(shapes)], [rnd(900 + i, *s) for i, s in enumerate(shapes)]
    flat = lambda ts: [t for x in ts for t in (x if x.dim() == 3 else [x])]
    refs = [ref64.muon(a, b, c, 0.02, 0.95, 0.01) for a, b, c in zip(flat(w), flat(g), flat(m))]
    import nvfp4_gemm_b200 as P
    P.pact_muon_step(w, g, m, lr=0.02, weight_decay=0.01)
    torch.cuda.synchronize()
    for a, c, (rm, rw) in zip(flat(w), flat(m), refs):
        ref64.within(c, rm, f"m {tuple(a.shape)}")
        ref64.within(a, rw, f"W {tuple(a.shape)}")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_that_are_not_finite_stay_with_their_matrix(bad):
    """The other matrices of the call, of the same batch and cluster too, are updated as without them."""
    import nvfp4_gemm_b200 as P
    w, g = [rnd(1, 6, 16, 200), rnd(2, 40, 16)], [rnd(3, 6, 16, 200), rnd(4, 40, 16)]
    runs = []
    for spoil in (False, True):
        w1, g1 = [t.clone() for t in w], [t.clone() for t in g]
        m1 = [torch.zeros_like(t) for t in w]
        if spoil:
            g1[0][2, 3, 7] = bad
        P.pact_muon_step(w1, g1, m1, lr=0.1)
        runs.append((w1, m1))
    torch.cuda.synchronize()
    (wa, ma), (wb, mb) = runs
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(wa[0][keep], wb[0][keep]) and torch.equal(ma[0][keep], mb[0][keep])
    assert torch.equal(wa[1], wb[1]) and torch.equal(ma[1], mb[1])
    assert bool(wb[0][2].isnan().all())
