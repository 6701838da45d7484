"""engram_fp8_quantise on rows of very many blocks of 128: more than 65,536, where a division
by a 32-bit reciprocal stops being exact.  Bytes and scales have one right answer (the smallest
power of two 2^e with the block's largest magnitude at most 448 * 2^e, values rounded to nearest
even), worked out in fp64 on the device."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def reference(x):
    """(values of the bytes, scale bytes) of x [M, K], a block at a time along K."""
    import torch
    M, K = x.shape
    blocks = torch.nn.functional.pad(x.double(), (0, -K % 128)).view(M, -1, 128)
    big = blocks.abs().amax(2)
    m, ex = torch.frexp(big / 448)  # big = 448 m 2^ex, 1/2 <= m < 1
    e = torch.where(big > 0, ex - (m == 0.5).to(ex.dtype), -127).clamp(min=-127).double()
    v = blocks * torch.exp2(-e).unsqueeze(2)
    _, ex = torch.frexp(v)
    step = torch.exp2((ex.double() - 1).clamp(min=-6) - 3)  # e4m3's grid at |v|
    return (torch.round(v / step) * step).view(M, -1)[:, :K], (e + 127).to(torch.uint8)


# kblocks 100,003 and 65,537 divide wrongly by ceil(2^32 / kblocks) at a row's last block, 65,536
# is the last width that cannot; 62 .. 65 lie around the widths where the split changes its form.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,kblocks,short", [(1, 100003, 5), (3, 100003, 5), (1, 100003, 0), (2, 65537, 127),
                                             (2, 65536, 3), (1, 140001, 64), (700, 62, 1), (700, 63, 9), (700, 64, 100),
                                             (700, 65, 60), (9, 15, 3), (9, 16, 3), (9, 17, 3), (3000, 1, 127),
                                             (9000, 2, 1), (40000, 3, 50)])
def test_every_block_of_a_row(eg, M, kblocks, short, dtype):
    import torch
    K = kblocks * 128 - short
    g = torch.Generator(device="cuda").manual_seed(kblocks + M)
    wide = torch.randn(M, K + 24, generator=g, device="cuda")  # with a gap: not the form for gapless rows
    e = torch.randint(-20, 20, (M, (K + 24) // 128 + 1), generator=g, device="cuda").float()
    wide *= torch.exp2(e).repeat_interleave(128, 1)[:, :K + 24]
    wide = wide.to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    for x in (wide[:, :K], wide[:, 3:3 + K]):  # rows on and off 16-byte boundaries
        stride = (K + 15) // 16 * 16 + 16
        buf = torch.full((M, stride), 7, dtype=torch.uint8, device="cuda")
        s = torch.full((M, kblocks), 77, dtype=torch.uint8, device="cuda")
        eg.engram_fp8_quantise(x, out=[buf[:, :K], s])
        want, scales = reference(x)
        assert torch.equal(s, scales)
        assert torch.equal(buf[:, :K].contiguous().view(torch.float8_e4m3fn).double(), want)
        assert (buf[:, K:] == 7).all()
