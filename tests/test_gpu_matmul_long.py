"""bf16 outputs of sums of millions: parts of at most 262,144 values, so that what the tensor cores cut
off stays under the output's own rounding.

All products are positive, so a part's accumulator grows to its sum and each of its 16,384 additions of
16 products cuts off less than one unit in the last place, 2^-23 of it: 16,384 2^-23 of the result at
most.  The parts are added to nearest (2^-24 each, some hundred at most): 2^-17.  The output rounds by
half a step, 2^-8.  In one accumulator 2^25 of K are 1.1e-2 off, past the 2e-3 + 4e-3 allowed."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def positive(g, rows, cols):
    """Values in [1/2, 1) of bf16, a slab at a time."""
    import torch
    t = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for c in range(0, cols, 1 << 22):
        v = t[:, c:c + (1 << 22)]
        v.copy_(torch.rand(v.shape, generator=g, device="cuda") * 0.498 + 0.5)
    return t


def exact(a, b):
    import torch
    total = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device="cuda")
    for c in range(0, a.shape[1], 1 << 20):
        total += a[:, c:c + (1 << 20)].double() @ b[:, c:c + (1 << 20)].double().t()
    return total


def near(got, want):
    off = float(((got.double() - want) / want).abs().max())
    assert off <= 16384 * 2.0 ** -23 + 2.0 ** -17 + 2.0 ** -8, off


@pytest.mark.parametrize("M,N,K", [(4, 16, 1 << 25), (40, 24, 1 << 22), (130, 40, 1 << 25), (300, 264, (1 << 23) + 77)])
def test_products(eg, M, N, K):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = positive(g, M, K), positive(g, N, K)
    near(eg.engram_matmul(a, b, out_dtype=torch.bfloat16), exact(a, b))


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_of_millions_of_tokens(eg, accumulate):
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 1 << 25, 72, 40
    y, a = positive(g, N, M), positive(g, K, M)
    b = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    want = exact(y, a)
    old = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    _, db, _ = eg.engram_matmul_grad(y.t().contiguous(), a.t(), b, grad_a=False, accumulate=accumulate,
                                     db=old if accumulate else None)
    near(db, want)
