"""A copy that never arrives: the bounded waits of every form of engram_matmul, of the gradient's
two products in one launch and of engram_orthogonalise run out, the launch ends by itself with
ENGRAM_FLAG_TIMEOUT and leaves its outputs unwritten, and the next launch on the same context is
right."""
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


@pytest.fixture
def withheld(eg):
    """Runs a call whose first launch withholds a copy; returns its status and flags."""
    import torch
    previous = eg.engram_set_wait_limit_ns(LIMIT_NS)

    def run(call):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        eg.engram_debug_withhold_copies(1)
        call(status)
        return eg.engram_read_status(status)
    try:
        yield run
    finally:
        eg.engram_debug_withhold_copies(0)
        eg.engram_set_wait_limit_ns(previous)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(64, 512, 4096),   # K shared by CTAs
                                   (300, 300, 640),   # single CTAs
                                   (300, 301, 640),   # values one by one
                                   (300, 300, 2048),  # segments of fp32 outputs
                                   (4096, 4096, 512), (4096, 4095, 512),  # pairs
                                   (4096, 1024, 2048)])
def test_matmul(eg, withheld, M, N, K, out):
    import torch
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    a, b = torch.randn(M, K, device="cuda").bfloat16(), torch.randn(N, K, device="cuda").bfloat16()
    x = torch.randn(M, N, device="cuda").to(dt)
    for residual in (None, x):
        want = eg.engram_matmul(a, b, residual=residual, out_dtype=dt)
        got, pre = (torch.full((M, N), 77.0, dtype=dt, device="cuda") for _ in range(2))
        assert withheld(lambda st: eg.engram_matmul(a, b, residual=residual, pre=pre, out=got, status=st)) == \
            (eg.ERR_TIMEOUT, eg.FLAG_TIMEOUT)
        assert (got == 77.0).all() and (pre == 77.0).all()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        eg.engram_matmul(a, b, residual=residual, out=got, status=status)
        assert eg.engram_read_status(status) == (eg.OK, 0)
        assert torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(300, 256, 520), (1000, 2048, 3000)])
def test_gradient(eg, withheld, M, N, K):
    import torch
    a, b, dy = (torch.randn(*s, device="cuda").bfloat16() for s in ((M, K), (N, K), (M, N)))
    want = eg.engram_matmul_grad(dy, a, b)
    got = [torch.full_like(t, 77.0) for t in want[:2]]
    assert withheld(lambda st: eg.engram_matmul_grad(dy, a, b, da=got[0], db=got[1], status=st)) == \
        (eg.ERR_TIMEOUT, eg.FLAG_TIMEOUT)
    assert any((t == 77.0).all() for t in got)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_matmul_grad(dy, a, b, da=got[0], db=got[1], status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("L,M,N", [(1, 256, 1536), (8, 1024, 1100), (2, 90, 100), (1, 60, 2000)])
def test_orthogonalise(eg, withheld, L, M, N):
    import torch
    g = torch.randn(L, M, N, device="cuda")
    want = eg.engram_orthogonalise(g)
    assert withheld(lambda st: eg.engram_orthogonalise(g, status=st)) == (eg.ERR_TIMEOUT, eg.FLAG_TIMEOUT)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(eg.engram_orthogonalise(g, status=status), want)
    assert eg.engram_read_status(status) == (eg.OK, 0)
