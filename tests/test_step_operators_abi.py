"""Refusals of the rotation, attention and update calls, without a GPU: the library's host checks
(nothing is enqueued) and the binding's."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def P():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("_pact_build", os.path.join(root, "nvfp4_gemm_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build()
    import nvfp4_gemm_b200 as p
    return p


INVALID, SHAPE, ALIGN = 1, 2, 3


def test_rope(P):
    freq = (ctypes.c_double * 64)()
    call = lambda x=0x1000, ldx=512, M=4, h=4, D=128, pos=0x2000, f=freq, y=0x3000, ldy=512: P.pact.lib.pact_rope(
        x, ldx, M, h, D, pos, f, 0, y, ldy, None)
    assert call(x=None) == call(pos=None) == call(y=None) == call(f=None) == INVALID
    assert call(D=96) == call(M=0) == call(h=0) == call(ldx=504) == call(ldy=504) == call(M=2 ** 31) == SHAPE
    assert call(x=0x1008) == call(y=0x3004) == call(ldx=516) == call(pos=0x2002) == ALIGN
    assert "aligned" in P.pact_last_error()


def attention(P, **kw):
    a = P.pact.c_attention(300, 8, 2, 64, 0.125, 0x1000, 512, 0x2000, 128, 0x3000, 128, 0x4000, 3)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


BAD = [(dict(q=None), INVALID), (dict(seq_start=None), INVALID), (dict(scale=float("nan")), INVALID),
       (dict(scale=-0.125), INVALID), (dict(scale=0.0), INVALID),
       (dict(head_dim=96), SHAPE), (dict(heads=7), SHAPE), (dict(heads=0), SHAPE), (dict(kv_heads=0), SHAPE),
       (dict(M=0), SHAPE), (dict(M=2 ** 30 + 1), SHAPE), (dict(nseq=0), SHAPE), (dict(ldq=504), SHAPE),
       (dict(ldk=120), SHAPE), (dict(ldv=120), SHAPE), (dict(q=0x1008), ALIGN), (dict(k=0x2002), ALIGN),
       (dict(v=0x3008), ALIGN), (dict(ldv=132), ALIGN), (dict(seq_start=0x4002), ALIGN)]


@pytest.mark.parametrize("kw,status", BAD, ids=lambda x: str(x))
def test_attention_arguments(P, kw, status):
    lib = P.pact.lib
    assert lib.pact_attention_fwd(attention(P, **kw), 0x5000, 512, 0x6000, None) == status
    g = P.pact.c_attention_grad(0x5000, 512, 0x6000, 0x7000, 512, 0x8000, 512, 0x9000, 128, 0xA000, 128)
    assert lib.pact_attention_bwd(attention(P, **kw), ctypes.byref(g), 0xB000, 1 << 30, None) == status


def test_attention_outputs(P):
    lib = P.pact.lib
    assert lib.pact_attention_fwd(None, 0x5000, 512, 0x6000, None) == INVALID
    assert lib.pact_attention_fwd(attention(P), None, 512, 0x6000, None) == INVALID
    assert lib.pact_attention_fwd(attention(P), 0x5000, 504, 0x6000, None) == ALIGN
    assert lib.pact_attention_fwd(attention(P), 0x5000, 512, 0x6004, None) == ALIGN
    need = P.pact_attention_bwd_workspace_bytes(300, 8)
    assert need > 0 and P.pact_attention_bwd_workspace_bytes(0, 8) == 0
    names = [f[0] for f in P.pact.c_attention_grad._fields_]
    good = (0x5000, 512, 0x6000, 0x7000, 512, 0x8000, 512, 0x9000, 128, 0xA000, 128)
    call = lambda ws=0xB000, n=need, **kw: lib.pact_attention_bwd(
        attention(P), ctypes.byref(P.pact.c_attention_grad(*[kw.get(k, v) for k, v in zip(names, good)])), ws, n, None)
    for name in ("o", "lse", "dout", "dq", "dk", "dv"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: 0x5008}) == ALIGN
    assert call(ws=None) == call(n=need - 1) == INVALID
    assert call(ws=0xB008) == call(lddk=120) == call(lddq=516) == ALIGN


def test_muon(P):
    lib, c = P.pact.lib, P.pact.c_muon_matrix
    good = [0x1000, 0x2000, 0x2000, 0x3000, 0x3000, 0x4000, 1, 16, 300]

    def call(n=1, ws=0x10000, size=None, lr=0.1, **at):
        m = (c * 2)(c(*good), c(*[at.get(f[0], v) for f, v in zip(c._fields_, good)]))
        need = lib.pact_muon_workspace_bytes(m, 2)
        return lib.pact_muon_step(m, 2 if n == 1 else n, 0, lr, 0.9, 0.0, 1, ws, need if size is None else size, None)
    for name in ("grad", "momentum", "momentum_out", "weight", "weight_out"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: 0x1001}) == ALIGN
    assert call(weight_bf16=0x4001) == ALIGN
    assert call(rows=65, cols=65) == call(rows=0) == call(cols=2 ** 24 + 1) == call(count=0) == SHAPE
    assert call(n=0) == call(ws=None) == call(size=8) == call(lr=float("inf")) == INVALID
    assert call(ws=0x10008) == ALIGN
    assert P.pact_muon_workspace_bytes([(65, 65)]) == 0 < P.pact_muon_workspace_bytes([(64, 65)])


def test_binding_refuses_host_tensors(P):
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        P.pact_rope(x, torch.zeros(4, dtype=torch.int32), [0.0] * 32, 2)
    with pytest.raises(TypeError):
        P.pact_attention_fwd(x, x, x, torch.zeros(2, dtype=torch.int32), 2, 2)
    with pytest.raises(TypeError):
        P.pact_muon_step([torch.zeros(4, 8)], [torch.zeros(4, 8)], [torch.zeros(4, 8)], lr=0.1)
    with pytest.raises(ValueError):
        P.pact_muon_step([], [], [], lr=0.1)


def test_packings_that_are_none_are_refused(P):
    from nvfp4_gemm_b200.layer import check_packing
    for good in ([0, 3, 3, 10], [2, 2, 2, 2], [0, 1, 2, 9]):
        check_packing(torch.tensor(good, dtype=torch.int32), 3, 10)
    for bad in ([0], [0, 3, 10], [0, 3, 2, 10], [0, 3, 3, 11], [-1, 3, 3, 10]):
        with pytest.raises(ValueError):
            check_packing(torch.tensor(bad, dtype=torch.int32), 3, 10)
    for bad in (torch.tensor(0), torch.zeros((2, 2)), torch.zeros(1)):
        with pytest.raises(ValueError):
            check_packing(bad, bad.numel() - 1, 10)


def test_overlapping_outputs_are_refused(P):
    """Matrices of one buffer may lie side by side (nothing below is refused for that alone: the last
    checks before the overlap are those of alignment, all of which pass)."""
    lib = P.pact.lib
    freq, base = (ctypes.c_double * 64)(), 0x100000
    rope = lambda y, ldy=1024: lib.pact_rope(base, 1024, 4, 4, 128, 0x2000, freq, 0, y, ldy, None)
    for y, ldy in ((base + 2 * 1024, 1024), (base + 2 * 504, 1024), (base - 2 * 8, 1024), (base, 512),
                   (base + 2 * 1024, 2048), (base + 2 * 528, 1024)):
        assert rope(y, ldy) == INVALID and "overlaps" in P.pact_last_error()
    # M = 300 rows of q (512 columns), k and v (128 each) in one buffer of rows of 768
    q, k, v = base, base + 2 * 512, base + 2 * 640
    a = lambda: attention(P, q=q, k=k, v=v, ldq=768, ldk=768, ldv=768)
    far = 0x800000
    for o, ldo in ((q, 768), (k, 768), (q + 2 * 768 * 299, 512), (v - 2 * 512, 768), (base - 2 * 8, 512)):
        assert lib.pact_attention_fwd(a(), o, ldo, 0x6000, None) == INVALID and "overlaps" in P.pact_last_error()
    names = [f[0] for f in P.pact.c_attention_grad._fields_]
    good = (far, 512, 0x6000, 2 * far, 512, 3 * far, 768, 3 * far + 1024, 768, 3 * far + 1280, 768)
    for at in (dict(dq=far), dict(dk=2 * far + 2 * 512), dict(dv=3 * far + 1024), dict(dq=q), dict(dv=v), dict(dk=3 * far + 1008),
               dict(dv=3 * far + 2 * 768 - 2 * 120)):
        g = P.pact.c_attention_grad(*[at.get(k, v) for k, v in zip(names, good)])
        assert lib.pact_attention_bwd(a(), ctypes.byref(g), 0xB000, 1 << 30, None) == INVALID
        assert "overlap" in P.pact_last_error(), at


def test_a_matrix_given_twice_is_refused(P):
    lib, c = P.pact.lib, P.pact.c_muon_matrix

    def call(*at):
        m = (c * len(at))(*[c(*a, 1, 16, 300) for a in at])
        return lib.pact_muon_step(m, len(at), 0, 0.1, 0.9, 0.0, 1, 0x10, lib.pact_muon_workspace_bytes(m, len(at)), None)
    size = 16 * 300 * 4
    one = [0x1000, 0x100000, 0x100000, 0x200000, 0x200000, 0x300000]
    for k in (2, 4, 5):   # the same momentum, weight or BF16 copy, and one that begins inside it
        for shift in (0, size // 2 - 4):
            other = [0x1000] + [p + size for p in one[1:]]
            other[k] = one[k] + shift
            assert call(one, other) == call(other, one) == INVALID and "twice" in P.pact_last_error()
    assert call([0x1000, 0x100000, 0x100000, 0x200000, 0x100000, None]) == INVALID


@pytest.mark.parametrize("fp32", [0, 1])
def test_an_update_over_its_inputs_is_refused(P, fp32):
    """But for a momentum or weight updated in place, no output may share memory with what the call reads."""
    lib, c = P.pact.lib, P.pact.c_muon_matrix
    rows, cols = 16, 300
    size, gsize = 4 * rows * cols, (4 if fp32 else 2) * rows * cols
    ws = 0x4000000

    def call(*at, ws=ws):
        m = (c * len(at))(*[c(*a, 1, rows, cols) for a in at])
        return lib.pact_muon_step(m, len(at), fp32, 0.1, 0.9, 0.0, 1, ws, lib.pact_muon_workspace_bytes(m, len(at)), None)
    #       grad      momentum  its output weight   its output BF16 copy
    one = [0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000]
    two = [p + 0x1000000 for p in one]
    # What is no overlap passes the check.  Only without a device, where the launch behind it fails: these
    # addresses are none of its memory.
    if not torch.cuda.is_available():
        for fine in ((one, two), ([one[0], one[1], one[1], one[3], one[3], one[5]], two), (one, [one[0]] + two[1:]),
                     (one, [two[0], one[1], two[2], one[3], *two[4:]])):
            assert call(*fine) != INVALID, P.pact_last_error()
    outs, ins = (2, 4, 5), (0, 1, 3)
    for o in outs:
        for i in ins:
            far = gsize if i == 0 else size
            for shift in (0, 16, far - 16):
                if shift == 0 and (o, i) in ((2, 1), (4, 3)):
                    continue                      # in place
                same, other = list(one), list(two)
                same[o] = one[i] + shift          # the entry's own input
                other[o] = one[i] + shift         # another entry's
                assert call(same, two) == INVALID and "overlap" in P.pact_last_error()
                assert call(one, other) == call(other, one) == INVALID
        at = list(two)
        at[o] = one[1]
        assert call(one, at) == INVALID           # another entry's momentum, whole
        assert call(one, two, ws=one[o] - 16) == INVALID
    for i in ins:
        assert call(one, two, ws=two[i] - 16) == INVALID


def test_statistics_and_scratch_over_other_memory_are_refused(P):
    """lse and the workspace are outputs like the others, and no output may lie over the row numbers."""
    lib = P.pact.lib
    M, hq, freq = 300, 8, (ctypes.c_double * 64)()
    at = {n: i << 20 for i, n in enumerate("q k v seq o lse dout dq dk dv ws".split(), 1)}
    a = lambda: attention(P, q=at["q"], k=at["k"], v=at["v"], ldq=768, ldk=768, ldv=768, seq_start=at["seq"])
    need = P.pact_attention_bwd_workspace_bytes(M, hq)

    def bwd(**kw):
        n = at | kw
        g = P.pact.c_attention_grad(n["o"], 512, n["lse"], n["dout"], 512, n["dq"], 512, n["dk"], 128, n["dv"], 128)
        return lib.pact_attention_bwd(a(), ctypes.byref(g), n["ws"], need, None)
    width = {"q": 512, "k": 128, "v": 128}
    for name in "qkv":
        last = at[name] + 2 * (299 * 768 + width[name]) - 16    # the last 16 bytes of the last row
        assert lib.pact_attention_fwd(a(), at["o"], 512, last, None) == INVALID and "overlap" in P.pact_last_error()
        assert bwd(ws=last) == INVALID and "overlap" in P.pact_last_error()
    assert lib.pact_attention_fwd(a(), at["o"], 512, at["o"] + 16, None) == INVALID
    assert lib.pact_attention_fwd(a(), at["o"], 512, at["seq"] - 4 * M * hq + 16, None) == INVALID
    assert lib.pact_attention_fwd(a(), at["seq"] - 16, 512, at["lse"], None) == INVALID
    for name in ("o", "lse", "dout", "dq", "dk", "dv", "seq"):
        assert bwd(ws=at[name] - need + 16) == INVALID and "overlap" in P.pact_last_error(), name
    for name in ("dq", "dk", "dv"):
        assert bwd(**{name: at["lse"]}) == bwd(**{name: at["seq"] - 16}) == INVALID
    assert lib.pact_rope(at["q"], 512, 4, 4, 128, at["o"] + 16, freq, 0, at["o"], 512, None) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would launch on addresses of no memory")
def test_overlaps_of_any_two_strides(P):
    """Refused exactly where two matrices share an element, against their enumeration."""
    import random
    lib, freq, base, D = P.pact.lib, (ctypes.c_double * 32)(), 0x1000000, 64
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(1500):
        M, ldx, ldy = rng.randint(1, 7), 8 * rng.randint(8, 40), 8 * rng.randint(8, 40)
        y = 8 * rng.randint(-7 * 40, 7 * 40)
        cells = lambda p, ld: {p + r * ld + c for r in range(M) for c in range(D)}
        share = bool(cells(0, ldx) & cells(y, ldy)) and not (y == 0 and (ldx == ldy or M == 1))
        got = lib.pact_rope(base, ldx, M, 1, D, 0x2000, freq, 0, base + 2 * y, ldy, None)
        assert (got == INVALID) == share, (M, ldx, ldy, y)
        seen[share] += 1
    assert min(seen) > 300


@pytest.mark.parametrize("starts,error", [([0, 2 ** 32, 2 ** 32 + 8], ValueError), ([0.0, 3.5, 8.0], TypeError),
                                          ([False, True, True], TypeError)], ids=str)
def test_a_packing_is_checked_before_it_is_cast(P, starts, error):
    """Row numbers that an int32 would hold wrapped or rounded; other whole numbers are as good as int32."""
    from types import SimpleNamespace

    from nvfp4_gemm_b200.layer import AttentionCore, LayerShape, PactLayer, check_packing
    check_packing(torch.tensor([0, 3, 8], dtype=torch.int16), 2, 10)
    starts = torch.tensor(starts)
    with pytest.raises(error):
        check_packing(starts, 2, 10)
    layer = SimpleNamespace(s=LayerShape(M=10, H=128, I=256, KV=64), attention=AttentionCore(64, starts, [0.0] * 32))
    with pytest.raises(error):
        PactLayer._init_attention(layer, "cpu")
