"""pact_rope against its 64-bit form: both head sizes and directions, few and many rows, far
positions, strides, padding rows, in place."""
import pytest
import torch

from tests import ref64

pytestmark = pytest.mark.gpu


def freqs(D, theta=5e5):
    return [theta ** (-2 * i / D) for i in range(D // 2)]


def bf(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("M,heads,D", [(1, 1, 64), (3, 5, 128), (130, 40, 64), (2371, 14, 128), (5000, 3, 64)])
def test_matches_the_64_bit_form(guards, M, heads, D, inverse):
    import nvfp4_gemm_b200 as P
    x = bf(M, M, heads * D + 16)[:, 8:8 + heads * D]
    pos = torch.randint(0, 1 << 20, (M,), device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    y = guards.matrix(M, heads * D, pad_cols=24)
    P.pact_rope(x, pos, freqs(D), heads, y=y, inverse=inverse)
    ref64.within(y, ref64.rope(x, pos, freqs(D), heads, inverse), "y")


def test_padding_rows_stay_and_in_place_is_the_same():
    import nvfp4_gemm_b200 as P
    M, heads, D = 77, 6, 64
    x = bf(1, M, heads * D)
    pos = torch.arange(M, device="cuda", dtype=torch.int32)
    pos[70:] = -1
    pos[3] = -5
    y = torch.full_like(x, 7.0)
    P.pact_rope(x, pos, freqs(D), heads, y=y)
    assert torch.equal(y[pos < 0], torch.full_like(y[pos < 0], 7.0))
    z = x.clone()
    assert P.pact_rope(z, pos, freqs(D), heads, y=z) is z
    assert torch.equal(z[pos < 0], x[pos < 0]) and torch.equal(z[pos >= 0], y[pos >= 0])


def test_inverse_is_the_transpose():
    """<rope(x), y> = <x, rope^T(y)>, up to the roundings of both (each output by H of its size)."""
    import nvfp4_gemm_b200 as P
    x, y = bf(5, 64, 256), bf(6, 64, 256)
    pos = torch.randint(0, 9000, (64,), device="cuda", dtype=torch.int32)
    a = P.pact_rope(x, pos, freqs(128), 2).double()
    b = P.pact_rope(y, pos, freqs(128), 2, inverse=True).double()
    tol = 1.1 * ref64.H * ((a * y).abs().sum() + (x * b).abs().sum())
    assert abs((a * y.double()).sum() - (x.double() * b).sum()) <= tol


def test_captured_and_on_another_stream():
    import nvfp4_gemm_b200 as P
    x, pos = bf(8, 300, 512), torch.arange(300, device="cuda", dtype=torch.int32)
    want = P.pact_rope(x, pos, freqs(64), 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = P.pact_rope(x, pos, freqs(64), 8)
    side.synchronize()
    assert torch.equal(got, want)
    y, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pact_rope(x, pos, freqs(64), 8, y=y)
    x.copy_(bf(9, 300, 512))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, P.pact_rope(x, pos, freqs(64), 8))


@pytest.mark.parametrize("heads,D", [(8, 65), (8, 129), (16, 127), (4, 96), (4, 32)])
def test_other_head_sizes_are_refused(heads, D):
    """Odd ones too: 65 columns a head are not heads of 64."""
    import nvfp4_gemm_b200 as P
    x, pos = bf(1, 4, heads * D), torch.arange(4, device="cuda", dtype=torch.int32)
    y = torch.full_like(x, 7.0)
    with pytest.raises(P.PactError):
        P.pact_rope(x, pos, [0.0] * (D // 2), heads, y=y)
    assert bool((y == 7.0).all())
