"""A wait that runs out in engram_orthogonalise's one-launch form: the launch ends by itself, out
stays unwritten by every CTA of the matrix -- in a cluster only the first CTA's wait runs out, and
the others, whose own waits end, write nothing either -- and the next call is right."""
import pytest

pytestmark = pytest.mark.gpu
LIMIT_NS = 5_000_000


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


# CTAs by themselves, and clusters of 2, 4 and 8; wide and tall.
@pytest.mark.parametrize("steps", [1, 5, 64])
@pytest.mark.parametrize("L,M,N", [(2, 90, 100), (3, 100, 90), (1, 100, 700), (2, 700, 128), (1, 1500, 64), (1, 60, 2000),
                                   (1, 2001, 61)])
def test_out_stays_unwritten(eg, L, M, N, steps):
    import torch
    g = torch.randn(L, M, N, generator=torch.Generator(device="cuda").manual_seed(M), device="cuda")
    option = dict(coefficients=(1.5, -0.5, 0.0), steps=steps)
    want = eg.engram_orthogonalise(g, **option)
    out = torch.full_like(want, 77.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    previous = eg.engram_set_wait_limit_ns(LIMIT_NS)
    try:
        eg.engram_debug_withhold_copies(1)
        eg.engram_orthogonalise(g, out=out, status=status, **option)
        assert eg.engram_read_status(status) == (eg.ERR_TIMEOUT, eg.FLAG_TIMEOUT)
    finally:
        eg.engram_debug_withhold_copies(0)
        eg.engram_set_wait_limit_ns(previous)
    assert (out == 77.0).all()
    status.zero_()
    eg.engram_orthogonalise(g, out=out, status=status, **option)
    assert eg.engram_read_status(status) == (eg.OK, 0) and torch.equal(out, want)
