"""A copy that never arrives: the bounded waits of engram_fp8_quantise's tiles and of every form
of engram_fp8_matmul run out, the launch ends by itself with ENGRAM_FLAG_TIMEOUT and leaves its
outputs unwritten, and the next launch on the same context is right."""
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
    """Runs a call whose launch withholds a copy; returns its status and flags."""
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(128, 128), (1000, 1000), (4000, 4096)])
def test_quantise(eg, withheld, M, K, dtype):
    import torch
    x = torch.randn(M, K, device="cuda").to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    want = eg.engram_fp8_quantise(x, cols=True)
    out = [torch.full(t.shape, 0x55, dtype=torch.uint8, device="cuda") for t in want]
    out = [eg.fp8_empty(*t.shape, "cuda").fill_(0x55) if i % 2 == 0 else t for i, t in enumerate(out)]
    assert withheld(lambda st: eg.engram_fp8_quantise(x, cols=True, out=out, status=st)) == \
        (eg.ERR_TIMEOUT, eg.FLAG_TIMEOUT)
    assert all((t == 0x55).all() for t in out)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_fp8_quantise(x, cols=True, out=out, status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(130, 300, 640),      # single CTAs
                                   (5000, 300, 8320),    # with several accumulators
                                   (16, 300, 2048), (2000, 300, 9000),  # K shared by 8 and by 4 CTAs
                                   (9000, 300, 2048),    # CTA pairs
                                   (5000, 1500, 8320)])  # with several accumulators
def test_matmul(eg, withheld, M, N, K, out):
    import torch
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    a, sa = eg.engram_fp8_quantise(torch.randn(M, K, device="cuda"))
    b, sb = eg.engram_fp8_quantise(torch.randn(N, K, device="cuda"))
    want = eg.engram_fp8_matmul(a, sa, b, sb, out_dtype=dt)
    got = torch.full((M, N), 77.0, dtype=dt, device="cuda")
    assert withheld(lambda st: eg.engram_fp8_matmul(a, sa, b, sb, out=got, status=st)) == \
        (eg.ERR_TIMEOUT, eg.FLAG_TIMEOUT)
    assert (got == 77.0).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_fp8_matmul(a, sa, b, sb, out=got, status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert torch.equal(got, want)
