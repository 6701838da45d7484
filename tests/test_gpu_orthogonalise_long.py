"""The update of matrices with tens of millions of rows: the sums of their squares are as long.

X = u / |u| is multiplied by a polynomial of A = X^T X only, so the iteration runs in fp64 on the small
square matrix and a sample of the rows is compared.  Allowed: what the header states, 4e-3 of the
norm for the iteration in fp16 and half a step of bf16, 2^-8 of each value, for the result (its rms is
1.7e-3).  A's diagonal, sums of 2^25 squares, in one accumulator is 1e-2 off."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


@pytest.mark.parametrize("M,N", [(1 << 25, 136), (1 << 20, 200), (1 << 18, 136), ((1 << 18) + 1, 136), (136, 3000000)])
def test_long_sides(eg, M, N):
    import torch
    a, b, c = 3.4445, -4.7750, 2.0315
    g = torch.randn(M, N, generator=torch.Generator(device="cuda").manual_seed(N), device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = eg.engram_orthogonalise(g, status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    tall = g if M > N else g.t()
    gram = torch.zeros(min(M, N), min(M, N), dtype=torch.float64, device="cuda")
    for r in range(0, max(M, N), 1 << 20):
        x = tall[r:r + (1 << 20)].double()
        gram += x.t() @ x
    norm = gram.diagonal().sum().sqrt()
    gram /= norm * norm
    eye = torch.eye(min(M, N), dtype=torch.float64, device="cuda")
    whole = eye
    for _ in range(5):
        p = a * eye + b * gram + c * gram @ gram
        gram, whole = p @ gram @ p, whole @ p
    rows = torch.randint(0, max(M, N), (20000,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    want = tall[rows].double() / norm @ whole
    got = (out if M > N else out.t())[rows].double()
    off = float((got - want).norm() / want.norm())
    assert off <= 4e-3 + 2.0 ** -8, off
