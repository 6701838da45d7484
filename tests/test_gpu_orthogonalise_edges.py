"""engram_orthogonalise at the ends of fp32: gradients whose squares overflow or vanish, eps of zero,
values that are not finite.

The update does not depend on the gradient's size, and a power of two goes through every step
without a rounding: the sums of squares, their root and the quotients scale exactly, so gradients
times 2^k (whose values stay normal numbers) have the bits of the plain ones."""
import pytest

pytestmark = pytest.mark.gpu
# In one launch by a CTA, wide and tall, and by clusters of 2 and 8; a chain of launches.
SIZES = [(3, 90, 70), (2, 70, 120), (1, 100, 700), (1, 60, 2000), (2, 300, 200), (1, 130, 515)]


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def gradients(L, M, N):
    import torch
    x = torch.randn(L, M, N, generator=torch.Generator(device="cuda").manual_seed(M), device="cuda")
    return torch.where(x.abs() < 2.0 ** -10, 2.0 ** -10, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,M,N", SIZES)
def test_any_size_of_gradient(eg, L, M, N, dtype):
    import torch
    x = gradients(L, M, N).to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    want = eg.engram_orthogonalise(x, eps=0.0)
    assert want.isfinite().all() and want.any()
    for k in (-115, -90, -70, -50, -30, 30, 60, 66, 100, 124):
        assert torch.equal(eg.engram_orthogonalise(x * 2.0 ** k, eps=0.0), want), k
        if k > 0:  # the usual eps is nothing beside them
            assert torch.equal(eg.engram_orthogonalise(x * 2.0 ** k), want), k


@pytest.mark.parametrize("L,M,N", SIZES)
def test_momentum_of_any_size(eg, L, M, N):
    import torch
    x, m = gradients(L, M, N), gradients(L, M, N).roll(1, -1)
    first, want = m.clone(), None
    want = eg.engram_orthogonalise(x, momentum=first, beta=0.5, eps=0.0)
    for k in (-100, 100, 120):
        moved = m * 2.0 ** k
        assert torch.equal(eg.engram_orthogonalise(x * 2.0 ** k, momentum=moved, beta=0.5, eps=0.0), want)
        assert torch.equal(moved, first * 2.0 ** k)


@pytest.mark.parametrize("eps", [0.0, 1e-7, 3e38])
@pytest.mark.parametrize("L,M,N", SIZES)
def test_zeros_stay_zero(eg, L, M, N, eps):
    import torch
    x = torch.zeros(L + 1, M, N, device="cuda")
    x[0] = gradients(1, M, N)[0]
    out = eg.engram_orthogonalise(x, eps=eps)
    assert not out[1:].any() and out[0].isfinite().all() and (eps > 1 or out[0].any())


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("L,M,N", SIZES + [(1, 1, 1), (1, 1, 40), (1, 40, 1)])
def test_what_is_not_finite_is_its_own_matrixs(eg, L, M, N, value):
    """All of the matrix is NaN, whatever the number of steps, and no other matrix."""
    import torch
    x = gradients(L + 1, M, N)
    want = eg.engram_orthogonalise(x)
    x[0, M // 2, N // 3] = float(value)
    for steps in (1, 5):
        out = eg.engram_orthogonalise(x, steps=steps)
        assert out[0].isnan().all()
    assert torch.equal(out[1:], want[1:])
