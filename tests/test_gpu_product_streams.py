"""engram_matmul, engram_matmul_grad and engram_orthogonalise on streams of the caller's, several at
once, in threads and in graphs that share a workspace: the same bits as one after the other on the
current stream."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


# A few rows, K shared by CTAs, single tiles, pairs; the last two with copies of their operands.
PRODUCTS = [(1, 513, 700), (37, 256, 2048), (200, 512, 128), (1500, 1100, 520), (130, 201, 99), (700, 301, 1027)]
# In one launch by a CTA and by clusters, and a chain of launches.
MATRICES = [(3, 60, 90), (2, 100, 1300), (1, 200, 333)]


def inputs(seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    products = [(rand(M, K).bfloat16(), rand(N, K).bfloat16(), rand(M, N).bfloat16(), rand(N)) for M, N, K in PRODUCTS]
    return products, [rand(*s) for s in MATRICES]


def calls(eg, args, stream=None):
    out = []
    for a, b, dy, bias in args[0]:
        out.append(eg.engram_matmul(a, b, bias, activation=eg.ACT_SILU, residual=dy, stream=stream))
        out += eg.engram_matmul_grad(dy, a, b, pre=dy, activation=eg.ACT_GELU, grad_bias=True, stream=stream)
    return out + [eg.engram_orthogonalise(g, stream=stream) for g in args[1]]


def same(got, want):
    import torch
    return [i for i, (a, b) in enumerate(zip(got, want, strict=True)) if not torch.equal(a, b)] == []


@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("late", ["side", "current"])
def test_results_do_not_meet_the_current_streams_memory(eg, kind, late):
    import torch
    args = inputs(1)
    want = [t.clone() for t in calls(eg, args)]
    sizes = {t.untyped_storage().nbytes() for t in want}
    sizes |= {eg.engram_orthogonalise_workspace_bytes(*s) for s in MATRICES}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.stream(s if late == "side" else torch.cuda.current_stream()):
            torch.cuda._sleep(20_000_000)
        for size in sizes:
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
        got = calls(eg, args, s if kind == "object" else s.cuda_stream)
        noise = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF) for size in sizes for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        torch.cuda.current_stream().wait_stream(s)
        assert same(got, want)
        del got, noise


def test_threads_on_streams_of_their_own(eg):
    """Every kind of kernel beside every other, with tensor memory of the same SMs to share."""
    import torch
    args = [inputs(10 + i) for i in range(4)]
    want = [[t.clone() for t in calls(eg, a)] for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = calls(eg, args[i])
                s.synchronize()
                if not same(got, want[i]):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_graphs_that_share_a_workspace(eg):
    """Captured with the same workspace, replayed in turn, with inputs that change in between."""
    import torch
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    args = inputs(20)

    def gradients():
        return [t for a, b, dy, _ in args[0]
                for t in eg.engram_matmul_grad(dy, a, b, pre=dy, activation=eg.ACT_RELU, grad_bias=True, workspace=ws)]

    def updates():
        return ([eg.engram_matmul(a, b, workspace=ws) for a, b, _, _ in args[0]] +
                [eg.engram_orthogonalise(g, workspace=ws) for g in args[1]])
    graphs, outs = [], []
    for run in (gradients, updates):
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run())
        graphs.append(graph)
    for seed in (21, 22, 23):
        products, matrices = inputs(seed)
        for mine, new in zip(args[0], products):
            for t, n in zip(mine, new):
                t.copy_(n)
        for mine, new in zip(args[1], matrices):
            mine.copy_(new)
        ws.fill_(0xFF)
        for graph in (*graphs, *graphs):
            graph.replay()
        torch.cuda.synchronize()
        assert same(outs[0], gradients()) and same(outs[1], updates())


def test_tensors_of_another_place_are_refused(eg):
    """Before anything is launched, with a stream given and without."""
    import torch
    a = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(eg.EngramError):
            eg.engram_matmul(a, a.cpu(), stream=stream)
        with pytest.raises(eg.EngramError):
            eg.engram_matmul(a, a, bias=torch.zeros(4), stream=stream)
        with pytest.raises(eg.EngramError):
            eg.engram_matmul_grad(torch.zeros(4, 4), a, a, stream=stream)
        with pytest.raises(eg.EngramError):
            eg.engram_orthogonalise(a, momentum=torch.zeros(4, 8), stream=stream)
        with pytest.raises(eg.EngramError):
            eg.engram_orthogonalise(a, workspace=torch.zeros(1 << 16, dtype=torch.uint8), stream=stream)
