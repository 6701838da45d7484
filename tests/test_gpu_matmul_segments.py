"""Long sums of fp32 outputs are added up in parts of at most 768 values, rounding to nearest between
them.

a's rows are one 1 among t = 2^-30 and b is ones, so a row's sum is 1 + (K - 1) t exactly.  The
tensor cores add 16 products at a time: 16 t = 2^-26 to an accumulator that holds the 1 is an
eighth of its last place (2^-23), and where the addition cuts off, nothing stays of it.  So what is
missing from the sum is at most t for every value in the same part as the 1.  Sums of t alone are
exact (multiples of 2^-30 under 2^-6, 24 bits).  Every addition to the sum that holds the 1, which
stays under 2, rounds to nearest: half a step, 2^-24.  Where tiles walk K there is one for each part
after the first, ceil(K / 768) and a few at most, or where CTAs share K no more than that and 16.
Where warps take up to 16 rows, K is in 16 sums, so ceil(K / 16 / 768) and 16 to join those:
  1 + (K - 1) t - got <= 768 t + (additions) 2^-24.
In one accumulator all of K t would be missing, with the warps' K t / 16."""
import pytest

pytestmark = pytest.mark.gpu
T = 2.0 ** -30


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def missing(eg, M, N, K, at, values=None):
    """What the sums lack at most; row m has its 1 at at + 8 m.  values: that many of t from the
    beginning on, the rest zeros."""
    import torch
    a = torch.full((M, K), T, dtype=torch.bfloat16, device="cuda")
    a[:, values or K:] = 0
    a[torch.arange(M, device="cuda"), (at + 8 * torch.arange(M, device="cuda")) % (values or K)] = 1.0
    out = eg.engram_matmul(a, torch.ones(N, K, dtype=torch.bfloat16, device="cuda"))
    return float((1 + ((values or K) - 1) * T - out.double()).abs().max()) / T


def bound(additions):
    return 768 + additions * 2.0 ** -24 / T


@pytest.mark.parametrize("M,N,K", [(1, 64, 70000), (3, 4096, 65536), (8, 33, 262144), (2, 16, 1 << 20), (11, 40, 70000),
                                   (16, 130, 90001)])
@pytest.mark.parametrize("at", [0, 5000])
def test_few_rows(eg, M, N, K, at):
    assert missing(eg, M, N, K, at) <= bound(-(-K // 16 // 768) + 16)


# K shared by 2 to 8 CTAs; single CTAs; pairs; with and without rows on 16 bytes.
@pytest.mark.parametrize("M,N,K", [(40, 140, 10000), (128, 128, 30000), (40, 140, 70000), (300, 1024, 40000),
                                   (300, 1023, 40000), (1300, 1100, 30000), (4096, 4096, 20000), (4096, 4095, 20000)])
def test_tiles(eg, M, N, K):
    assert missing(eg, M, N, K, 64) <= bound(-(-K // 768) + 16)


@pytest.mark.parametrize("M,N,K", [(37, 4608, 16000), (20, 4608, 16384), (64, 4096, 15000), (100, 4096, 6144),
                                   (100, 4096, 16384)])
def test_shared_by_clusters(eg, M, N, K):
    """1024 values of K, those that the first of 4 CTAs once put into one accumulator: two parts of
    them at least, and only additions of those round."""
    assert missing(eg, M, N, K, 0, values=1024) <= bound(2)
