"""Packed causal attention and its gradient against their 64-bit forms, and what the calls
promise beside the numbers: isolation of sequences, untouched rows, streams, graphs, repeats."""
import math

import pytest
import torch

from tests import ref64

pytestmark = pytest.mark.gpu

# (sequence lengths, rows behind the last one, heads, key heads, head size)
CASES = [
    ([1], 0, 1, 1, 64),
    ([1], 0, 1, 1, 128),
    ([2, 0, 1, 0], 3, 3, 1, 128),
    ([127, 128, 129], 0, 4, 4, 64),
    ([127, 128, 129], 5, 4, 2, 128),
    ([64, 65, 1, 63], 0, 6, 2, 64),
    ([255, 256, 257], 1, 3, 1, 128),
    ([0, 0, 300, 0], 200, 5, 1, 64),
    ([1, 700, 2, 33], 130, 8, 2, 128),
    ([1023], 0, 12, 2, 128),
    ([513, 511], 0, 32, 8, 64),
    ([3] * 70 + [130], 0, 4, 1, 128),
    ([200, 0, 1] * 20, 11, 3, 1, 64),
    ([7, 300, 129, 2] * 8, 0, 2, 2, 128),
    ([260] + [0] * 40, 0, 5, 5, 64),
    ([1100, 5, 900], 43, 7, 7, 64),
]
IDS = [f"{len(c[0])}seq-{sum(c[0])}+{c[1]}-h{c[2]}k{c[3]}d{c[4]}" for c in CASES]


def bf(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def starts_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def problem(lens, pad, hq, hk, D, seed=0, std=1.0):
    starts = starts_of(lens)
    M = starts[-1] + pad
    qkv = bf(seed, M, (hq + 2 * hk) * D, std=std)
    return (qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D], qkv[:, (hq + hk) * D:],
            torch.tensor(starts, dtype=torch.int32, device="cuda"), starts, M)


def status_ok():
    import nvfp4_gemm_b200 as P
    assert P.pact_get_device_status() == 0, P.pact_last_error()


@pytest.mark.parametrize("lens,pad,hq,hk,D", CASES, ids=IDS)
def test_forward(guards, lens, pad, hq, hk, D):
    import nvfp4_gemm_b200 as P
    q, k, v, cu, starts, M = problem(lens, pad, hq, hk, D)
    o, lse = guards.matrix(M, hq * D, pad_cols=8), guards.flat(4 * hq * M).view(torch.float32).view(hq, M)
    before = o.clone()
    P.pact_attention_fwd(q, k, v, cu, hq, hk, o=o, lse=lse)
    status_ok()
    ref = ref64.attention(q, k, v, starts, hq, hk, D ** -0.5)
    n = starts[-1]
    ref64.within(o[:n], tuple(t[:n] for t in ref["o"]), "o")
    ref64.within(lse[:, :n], tuple(t[:, :n] for t in ref["lse"]), "lse")
    assert torch.equal(o[n:].view(torch.int16), before[n:].view(torch.int16)), "rows of no sequence were written"


@pytest.mark.parametrize("lens,pad,hq,hk,D", CASES, ids=IDS)
def test_gradient(guards, lens, pad, hq, hk, D):
    import nvfp4_gemm_b200 as P
    q, k, v, cu, starts, M = problem(lens, pad, hq, hk, D)
    do = bf(1, M, hq * D)
    ref = ref64.attention(q, k, v, starts, hq, hk, D ** -0.5)
    o, lse = ref["o"][0].bfloat16(), ref["lse"][0].float()
    outs = [guards.matrix(M, n * D, pad_cols=8) for n in (hq, hk, hk)]
    before = [t.clone() for t in outs]
    P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk, dq=outs[0], dk=outs[1], dv=outs[2])
    status_ok()
    ref = ref64.attention(q, k, v, starts, hq, hk, D ** -0.5, do, o)
    n = starts[-1]
    for name, t, b in zip(("dq", "dk", "dv"), outs, before):
        ref64.within(t[:n], tuple(x[:n] for x in ref[name]), name)
        assert torch.equal(t[n:].view(torch.int16), b[n:].view(torch.int16)), f"{name}: rows of no sequence written"


@pytest.mark.parametrize("D", [64, 128])
def test_gradient_against_differences(D):
    """f = <do, attention(q, k, v)> changes along a direction by the gradient's product with it; the
    differences are taken in 64 bits on the 64-bit form."""
    import nvfp4_gemm_b200 as P
    lens, hq, hk = [50, 1, 149], 4, 2
    q, k, v, cu, starts, M = problem(lens, 0, hq, hk, D)
    do = bf(3, M, hq * D)
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    grads = P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk)
    ref = ref64.attention(q, k, v, starts, hq, hk, D ** -0.5, do, o)
    f = lambda *t: (ref64.attention(*t, starts, hq, hk, D ** -0.5)["o"][0] * do.double()).sum().item()
    base = [t.double() for t in (q, k, v)]
    for i, (name, t) in enumerate(zip(("dq", "dk", "dv"), grads)):
        d = torch.randn(t.shape, generator=torch.Generator(device="cuda").manual_seed(7 + i), device="cuda",
                        dtype=torch.float64)
        e = 1e-4
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + e * d, base[i] - e * d
        slope = (f(*up) - f(*down)) / (2 * e)
        # the element bounds, plus o's rounding in delta (H |do . o| P per pair, random in sign: its
        # bound is the element bound again) and the differences' own e^2 term
        tol = 2 * (ref[name][1] * d.abs()).sum().item() + 1e-3 * abs(slope)
        assert abs((t.double() * d).sum().item() - slope) <= tol, name


@pytest.mark.parametrize("D", [64, 128])
def test_large_scores_and_ragged_strides(guards, D):
    """Scores up to some hundreds (the running maximum moves far), q, k, v and o in buffers of their own
    strides, a scale of its own."""
    import nvfp4_gemm_b200 as P
    lens, hq, hk = [333, 90], 6, 3
    starts = starts_of(lens)
    M = starts[-1]
    q, k, v = (bf(s, M, n * D + p, std=w)[:, p:] for s, n, p, w in ((1, hq, 8, 6), (2, hk, 24, 6), (3, hk, 40, 1)))
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    o = guards.matrix(M, hq * D, pad_cols=16)
    _, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk, scale=0.31, o=o)
    do = bf(4, M, hq * D)
    ref = ref64.attention(q, k, v, starts, hq, hk, 0.31, do, o)
    ref64.within(o, ref["o"], "o")
    ref64.within(lse, ref["lse"], "lse")
    for name, t in zip(("dq", "dk", "dv"), P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk, scale=0.31)):
        ref64.within(t, ref[name], name)
    status_ok()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128])
def test_sequences_do_not_reach_one_another(D, poison):
    """Values that are not finite, in other sequences and in rows of none (inputs, o, lse and do alike),
    change no bit of a sequence's results."""
    import nvfp4_gemm_b200 as P
    lens, pad, hq, hk = [130, 77, 200, 20], 60, 6, 2
    q, k, v, cu, starts, M = problem(lens, pad, hq, hk, D)
    do = bf(5, M, hq * D)
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    grads = P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk)
    bad = [slice(starts[1], starts[2]), slice(starts[3], M)]
    good = torch.cat([torch.arange(starts[0], starts[1]), torch.arange(starts[2], starts[3])]).cuda()
    q2, k2, v2, do2, o2, lse2 = (t.clone() for t in (q, k, v, do, o, lse))
    for rows in bad:
        for t in (q2, k2, v2, do2):
            t[rows] = poison
    o3, lse3 = P.pact_attention_fwd(q2, k2, v2, cu, hq, hk)
    assert torch.equal(o3[good], o[good]) and torch.equal(lse3[:, good], lse[:, good])
    for rows in bad:
        o2[rows] = poison
        lse2[:, rows] = poison
    for a, b in zip(P.pact_attention_bwd(do2, q2, k2, v2, o2, lse2, cu, hq, hk), grads):
        assert torch.equal(a[good], b[good])
    status_ok()


def test_repeats_agree_and_shared_workspaces_hold():
    """Every sum has a fixed order: calls agree bit for bit, eager and captured, and two captured calls
    that share a workspace replay in turn."""
    import nvfp4_gemm_b200 as P
    lens, hq, hk, D = [600, 3, 421], 8, 2, 128
    q, k, v, cu, starts, M = problem(lens, 0, hq, hk, D)
    dos = [bf(6, M, hq * D), bf(7, M, hq * D)]
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    want = [P.pact_attention_bwd(d, q, k, v, o, lse, cu, hq, hk) for d in dos]
    ws = torch.empty(P.pact_attention_bwd_workspace_bytes(M, hq), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for d in dos:
        outs.append([torch.zeros_like(t) for t in want[0]])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            o2, lse2 = P.pact_attention_fwd(q, k, v, cu, hq, hk)
            P.pact_attention_bwd(d, q, k, v, o2, lse2, cu, hq, hk, dq=outs[-1][0], dk=outs[-1][1], dv=outs[-1][2],
                                 workspace=ws)
    for i in (0, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # a captured call reads the row numbers anew at every replay
    cu.copy_(torch.tensor([0, 100, 100, M], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    assert all(torch.equal(a, b) for a, b in zip(outs[0], P.pact_attention_bwd(dos[0], q, k, v, o, lse, cu, hq, hk)))


@pytest.mark.parametrize("own_workspace", [True, False])
def test_two_streams_at_once(own_workspace):
    """With a workspace per call, and with the call's own (freed while its stream may still use it)."""
    import nvfp4_gemm_b200 as P
    D, hq, hk = 64, 8, 4
    jobs = []
    for i, lens in enumerate(([700, 9], [40] * 30)):
        q, k, v, cu, starts, M = problem(lens, 0, hq, hk, D, seed=i)
        do = bf(20 + i, M, hq * D)
        o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
        jobs.append(((do, q, k, v, o, lse, cu, hq, hk), P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got, held = [], []
    for _ in range(4):
        for s, (args, _) in zip(streams, jobs):
            ws = torch.empty(P.pact_attention_bwd_workspace_bytes(args[1].shape[0], hq), dtype=torch.uint8,
                             device="cuda") if own_workspace else None
            held.append(ws)
            got.append(P.pact_attention_bwd(*args, stream=s, workspace=ws))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, jobs[i % 2][1]))


def test_row_numbers_outside_the_rows_are_clamped():
    """seq_start beyond [0, M] is taken as the nearest end: no access leaves the rows."""
    import nvfp4_gemm_b200 as P
    q, k, v, cu, starts, M = problem([100, 60], 0, 4, 2, 64)
    want, _ = P.pact_attention_fwd(q, k, v, cu, 4, 2)
    wide = torch.tensor([-50, 100, 4000], dtype=torch.int32, device="cuda")
    got, _ = P.pact_attention_fwd(q, k, v, wide, 4, 2)
    assert torch.equal(got, want)
    status_ok()


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^32."""
    import nvfp4_gemm_b200 as P
    D, hq, hk, ld, n = 64, 2, 1, 65536, 150
    M = 2 ** 32 // ld + 200
    buf = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    starts = [M - n, M]
    buf[M - n:, :(hq + 2 * hk) * D] = bf(1, n, (hq + 2 * hk) * D)
    q, k, v = buf[:, :hq * D], buf[:, hq * D:(hq + hk) * D], buf[:, (hq + hk) * D:(hq + 2 * hk) * D]
    o = buf[:, 1024:1024 + hq * D]
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    _, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk, o=o)
    do, dq = buf[:, 2048:2048 + hq * D], buf[:, 4096:4096 + hq * D]
    do[M - n:] = bf(2, n, hq * D)
    _, dk, dv = P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk, dq=dq)
    tail = [t[M - n:] for t in (q, k, v)]
    ref = ref64.attention(*tail, [0, n], hq, hk, D ** -0.5, do[M - n:], o[M - n:])
    for name, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref64.within(t[M - n:], ref[name], name)
    status_ok()


@pytest.mark.parametrize("hq,hk,D", [(4, 2, 64), (3, 1, 128)])
def test_many_sequences_between_padding(hq, hk, D):
    """Over 32 sequences, with rows of none ahead of the first and behind the last: as the same sequences
    without them, and those rows left as they were."""
    import nvfp4_gemm_b200 as P
    lens, ahead, behind = [5, 0, 131, 64] * 10, 333, 77
    q, k, v, cu, starts, M = problem(lens, 0, hq, hk, D)
    do = bf(5, M, hq * D)
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    want = (o, *P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk))
    rows = slice(ahead, ahead + M)

    def wide(t):
        out = torch.full((ahead + M + behind, t.shape[1]), math.nan, dtype=t.dtype, device="cuda")
        out[rows] = t
        return out
    q2, k2, v2, do2 = wide(q), wide(k), wide(v), wide(do)
    outs = [torch.full_like(t, -7.0) for t in (q2, q2, k2, v2)]
    lse2 = torch.full((hq, ahead + M + behind), -7.0, device="cuda")
    P.pact_attention_fwd(q2, k2, v2, cu + ahead, hq, hk, o=outs[0], lse=lse2)
    P.pact_attention_bwd(do2, q2, k2, v2, outs[0], lse2, cu + ahead, hq, hk, dq=outs[1], dk=outs[2], dv=outs[3])
    status_ok()
    assert torch.equal(lse2[:, rows], lse)
    for got, ref in zip(outs, want):
        assert torch.equal(got[rows], ref)
        assert bool((got[:ahead] == -7.0).all() and (got[ahead + M:] == -7.0).all())
    assert bool((lse2[:, :ahead] == -7.0).all() and (lse2[:, ahead + M:] == -7.0).all())


@pytest.mark.parametrize("at", [0, 1, 5, 16, 17, 31, 144])
@pytest.mark.parametrize("lens", [[1], [1, 40, 200]], ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_a_query_that_is_not_finite_shows_in_its_gradients(D, lens, at):
    """A NaN in one query row: its own dq, and dk and dv of every key it sees, are NaN wherever it lies in
    its tile; the other sequences stay finite."""
    import nvfp4_gemm_b200 as P
    hq, hk, head = 4, 2, 1
    q, k, v, cu, starts, M = problem(lens, 0, hq, hk, D)
    do = bf(2, M, hq * D)
    a, b = starts[-2], M          # the last sequence
    row = a + min(at, b - a - 1)
    q[row, head * D] = math.nan
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    own, group = slice(head * D, (head + 1) * D), slice(0, D)
    assert bool(o[row, own].isnan().all() and lse[head, row].isnan())
    dq, dk, dv = P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk)
    status_ok()
    assert bool(dq[row, own].isnan().all()), "dq"
    for name, t in (("dk", dk), ("dv", dv)):
        assert bool(t[a:row + 1, group].isnan().all()), name
        assert bool(t[:a].isfinite().all() and t[:, D:].isfinite().all()), name


# Few rows under large groups: the gradients of k and v spread a key tile's heads over clusters of eight.
GROUPS = [([1], 0, 24, 1, 128), ([130, 5], 0, 24, 1, 128), ([700], 0, 24, 1, 128), ([260, 0, 1], 9, 9, 1, 128),
          ([127], 1, 16, 2, 128), ([400, 3], 0, 8, 1, 128), ([1], 0, 32, 1, 64), ([130, 5], 3, 32, 1, 64),
          ([513], 0, 9, 1, 64), ([90] * 40, 0, 8, 1, 64)]


@pytest.mark.parametrize("lens,pad,hq,hk,D", GROUPS, ids=[f"{len(c[0])}seq-{sum(c[0])}-h{c[2]}k{c[3]}d{c[4]}" for c in GROUPS])
def test_large_groups(guards, lens, pad, hq, hk, D):
    test_forward(guards, lens, pad, hq, hk, D)
    test_gradient(guards, lens, pad, hq, hk, D)


@pytest.mark.parametrize("D", [64, 128])
def test_scores_up_to_the_documented_size(D):
    """Scores of some 2^29, all apart by far more than an exponent: each row is its best key's v, off by the
    roundings of P and of o, and its log-sum that key's score."""
    import nvfp4_gemm_b200 as P
    n, size = 300, 2.0 ** 15
    g = torch.Generator(device="cuda").manual_seed(9)
    weight = (torch.randperm(256, generator=g, device="cuda")[torch.arange(n, device="cuda") % 256] - 128).double() / 128
    q, k = (torch.zeros((n, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[:, 0], k[:, 0] = size, (weight * size / 2).bfloat16()
    v = bf(10, n, D)
    cu = torch.tensor([0, 256], dtype=torch.int32, device="cuda")     # one key of each weight
    o, lse = P.pact_attention_fwd(q, k, v, cu, 1, 1, scale=1.0)
    status_ok()
    best = torch.cummax(k[:256, 0].double(), 0)
    want = v[:256].double()[best.indices]
    assert bool(((o[:256].double() - want).abs() <= 2.1 * ref64.H * want.abs() + ref64.T).all())
    assert bool(((lse[0, :256].double() - best.values * size).abs() <= 4 * ref64.U * best.values.abs() * size + 1).all())


@pytest.mark.parametrize("at", [0, 1, 17, 130])
@pytest.mark.parametrize("which", ["k", "v", "do"])
@pytest.mark.parametrize("D", [64, 128])
def test_keys_values_and_output_gradients_that_are_not_finite_show(D, which, at):
    """A NaN enters every result that the formula takes it into, and no other sequence's."""
    import nvfp4_gemm_b200 as P
    lens, hq, hk, head, col = [40, 200], 4, 2, 2, 5     # heads 2 and 3 read key head 1
    q, k, v, cu, starts, M = problem(lens, 0, hq, hk, D)
    do = bf(2, M, hq * D)
    a, group = lens[0], slice(D, 2 * D)
    {"k": k[:, group], "v": v[:, group], "do": do[:, head * D:(head + 1) * D]}[which][a + at, col] = math.nan
    o, lse = P.pact_attention_fwd(q, k, v, cu, hq, hk)
    dq, dk, dv = P.pact_attention_bwd(do, q, k, v, o, lse, cu, hq, hk)
    status_ok()
    nan = lambda t: bool(t.isnan().all())
    own = slice(head * D, (head + 1) * D)
    later, seen = slice(a + at, M), slice(a, a + at + 1)     # rows that see key `at`; keys that row `at` sees
    if which == "k":
        assert nan(lse[head, later]) and nan(o[later, own]) and nan(dq[later, own])
        assert nan(dk[a:, group]) and nan(dv[a:, group])     # the last row, of no log-sum, sees them all
    elif which == "v":
        assert nan(o[later, own][:, col]) and nan(dq[later, own]) and nan(dk[a:, group])
        assert bool(lse.isfinite().all())
    else:
        assert nan(dq[a + at, own]) and nan(dk[seen, group]) and nan(dv[seen, group][:, col])
    for t in (o, dq, dk, dv, lse.T):
        assert bool(t[:a].isfinite().all())
