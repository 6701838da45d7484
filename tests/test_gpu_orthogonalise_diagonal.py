"""The update of matrices with few rows or columns, whose square matrices are nearly diagonal: their
diagonals are not rounded to fp16.

`rounded` is the iteration in fp64 with the roundings that the kernels make: X and the square
matrices without their diagonals to fp16 times 2^8.  E is its distance from the iteration without any, R
the rounding of the result to bf16, both over a batch of 18 matrices.  The kernel's roundings fall on sums
that differ by fp32 rounding, so its error is another draw: of at least 18 * 16 * 16 roundings a step,
whose squares' mean is within 5 % in all but one of a thousand draws; 1.15 sqrt(E^2 + R^2) is allowed.
With the diagonals rounded it is 1.3 sqrt(E^2 + R^2)."""
import pytest

pytestmark = pytest.mark.gpu
A, B, C = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def half(t):
    return (t * 256).half().double() / 256


def iterate(u, rounded):
    import torch
    x = u / u.square().sum((1, 2), keepdim=True).sqrt()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = half(x) if rounded else x
    for step in range(5):
        gram = x @ x.transpose(1, 2)
        d = torch.diag_embed(gram.diagonal(dim1=1, dim2=2))
        gram = half(gram - d) + d if rounded else gram
        q = B * gram + C * (gram @ gram)
        e = torch.diag_embed(q.diagonal(dim1=1, dim2=2))
        q = half(q - e) + e if rounded else q
        x = A * x + q @ x
        x = half(x) if rounded and step < 4 else x
    return x.transpose(1, 2) if tall else x


def compare(eg, L, M, N, allowed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + 2 * N)
    u = torch.randn(L, M, N, generator=g, device="cuda")
    out = eg.engram_orthogonalise(u, eps=0.0).double()
    want = iterate(u.double(), False)
    E = float((iterate(u.double(), True) - want).norm())
    R = float((want.bfloat16().double() - want).norm())
    off = float((out - want).norm())
    assert off <= allowed * (E * E + R * R) ** 0.5, (off / (E * E + R * R) ** 0.5, off / float(want.norm()))


# By a CTA, wide and tall, and by clusters of 2, 4 and 8.
@pytest.mark.parametrize("M,N", [(16, 400), (400, 16), (20, 700), (23, 384), (384, 23), (64, 1000), (1000, 64), (40, 3000),
                                 (3000, 17)])
def test_nearly_diagonal(eg, M, N):
    compare(eg, 18, M, N, 1.15)


# By a chain of launches: its products by pairs, single CTAs and CTAs that share K, on rows or columns of out
# in the lanes, whole or on one side of the diagonal; out on 16 bytes and off them.
@pytest.mark.parametrize("L,M,N", [(20, 40, 3000), (20, 3000, 40), (2, 33, 6000), (1, 5001, 40), (3, 129, 4000), (3, 4000, 130),
                                   (1, 160, 6001), (2, 475, 5888), (1, 5888, 475), (4, 512, 6144), (1, 1024, 6144),
                                   (1, 6144, 1030), (24, 136, 2000)])
def test_nearly_diagonal_by_a_chain(eg, L, M, N):
    compare(eg, L, M, N, 1.15)


@pytest.mark.parametrize("L,M,N", [(2, 60, 90), (2, 300, 500), (2, 500, 300), (1, 700, 700)])
def test_a_coefficient_of_zero(eg, L, M, N):
    """c = 0: the diagonals go on without the square's part."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    u = torch.randn(L, M, N, generator=g, device="cuda")
    x = u.double() / u.double().square().sum((1, 2), keepdim=True).sqrt()
    for _ in range(6):
        x = 1.5 * x - 0.5 * (x @ x.transpose(1, 2) @ x)
    out = eg.engram_orthogonalise(u, steps=6, coefficients=(1.5, -0.5, 0.0), eps=0.0).double()
    assert float((out - x).norm() / x.norm()) <= 2.0 ** -8
