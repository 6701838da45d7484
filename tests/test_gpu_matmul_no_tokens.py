"""The gradient of no tokens zeroes db at every stride that the call takes: one row, whose stride
means nothing, rows side by side, rows with gaps and rows further apart than 2^31 bytes."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


@pytest.mark.parametrize("db", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,stride", [(1, 40, 0), (1, 40, 3), (1, 40, 64), (5, 40, 40), (5, 40, 47), (3, 40, 2 ** 30 + 24)])
def test_db_of_no_tokens(eg, N, K, stride, db):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[db]
    elements = (N - 1) * stride + K + 8
    flat = torch.full((elements,), 7.0, dtype=dt, device="cuda")
    grad = flat.as_strided((N, K), (stride, 1))
    a, b = torch.zeros(0, K, dtype=torch.bfloat16, device="cuda"), torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(0, N, dtype=torch.bfloat16, device="cuda")
    dbias = torch.full((N,), 7.0, device="cuda")
    eg.engram_matmul_grad(dy, a, b, db=grad, grad_bias=True, dbias=dbias)
    assert not grad.any() and not dbias.any()
    grad.fill_(7.0)
    assert (flat[:K + 8] == 7.0).all() and (flat[-K - 8:] == 7.0).all()
    if stride < 100:
        assert (flat == 7.0).all()
    eg.engram_matmul_grad(dy, a, b, db=grad, accumulate=True)
    assert (grad == 7.0).all()


@pytest.mark.parametrize("N,K,stride", [(1, 40, 0), (1, 40, 3), (5, 40, 47), (3, 40, 2 ** 30 + 24)])
def test_captured(eg, N, K, stride):
    import torch
    flat = torch.full(((N - 1) * stride + K,), 7.0, device="cuda")
    grad = flat.as_strided((N, K), (stride, 1))
    a, b = torch.zeros(0, K, dtype=torch.bfloat16, device="cuda"), torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(0, N, dtype=torch.bfloat16, device="cuda")
    eg.engram_matmul_grad(dy, a, b, db=grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.engram_matmul_grad(dy, a, b, db=grad)
    grad.fill_(7.0)
    graph.replay()
    assert not grad.any()
