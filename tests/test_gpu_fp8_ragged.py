"""engram_fp8_matmul where a warp of the epilogue has lanes past the last column of out, in every
form of the kernel: small whole numbers, whose sums are exact in fp32, so every output has one
right value and nothing beside out may change."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def operand(eg, rows, K, seed):
    """Whole numbers -3 .. 3 as e4m3 bytes with scales of 1 and 2, and their values in fp64."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-3, 4, (rows, K), generator=g, device="cuda").double()
    e = torch.randint(0, 2, (rows, -(-K // 128)), generator=g, device="cuda")
    q = eg.fp8_empty(rows, K, "cuda")
    q.copy_(v.float().to(torch.float8_e4m3fn).view(torch.uint8))
    return q, (e + 127).to(torch.uint8), v * torch.exp2(e.double()).repeat_interleave(128, 1)[:, :K]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 31, 33, 63, 97, 127, 129, 255, 257, 300])
@pytest.mark.parametrize("M,K", [(5, 200), (130, 640), (9000, 512),  # single CTAs
                                 (5000, 8320),                        # with several accumulators
                                 (16, 2048), (700, 8320),             # K shared by a cluster
                                 (20000, 4096),                       # CTA pairs, from 129 columns on
                                 (20000, 8320)])                      # with several accumulators
def test_columns_past_the_last(eg, M, N, K, out):
    import torch
    a, sa, av = operand(eg, M, K, M)
    b, sb, bv = operand(eg, N, K, N)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    buf = torch.full((M, N + 5), 77.0, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_fp8_matmul(a, sa, b, sb, out=buf[:, 2:2 + N], status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert torch.equal(buf[:, 2:2 + N], (av @ bv.t()).to(dt))
    assert (buf[:, :2] == 77.0).all() and (buf[:, 2 + N:] == 77.0).all()
