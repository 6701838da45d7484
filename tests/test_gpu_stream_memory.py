"""Calls on a side stream that make their own results and scratch, while the current stream
allocates and overwrites memory of the same sizes: the same bits as on the current stream."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def inputs():
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    T, R, D, rows = 9000, 2, 64, 700
    ids = torch.randint(0, rows, (T, R), generator=g, device="cuda", dtype=torch.int32)
    dy = torch.randn(T, R, D, generator=g, device="cuda")
    x = torch.randn(T, 4, 128, generator=g, device="cuda").bfloat16()
    k = torch.randn(T, 128, generator=g, device="cuda")
    return ids, dy, rows, x, k, torch.randn(4, generator=g, device="cuda"), x.flip(0).contiguous(), k[:rows].clone()


def calls(eg, args, stream):
    ids, dy, rows, x, k, alpha, dys, table = args
    out = [eg.engram_embed_grad(ids, dy, rows, stream=stream)]
    row_ids, grads, count = eg.engram_embed_grad_rows(ids, dy, rows, stream=stream)
    out += [row_ids, grads, count]
    out += eg.engram_gate_add_grad(k, None, x, alpha, dys, stream=stream)
    q = eg.engram_fp8_quantise(k, cols=True, stream=stream)
    out += list(q) + [eg.engram_fp8_matmul(q[0], q[1], q[0], q[1], stream=stream)]
    out += [eg.engram_embed(ids, table, stream=stream)]
    return out


@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("late", ["side", "current"])
def test_results_do_not_meet_the_current_streams_memory(eg, kind, late):
    """The side stream late: its kernels run after the current stream has written what it
    allocated since.  The current stream late: its writes into memory that it has freed by
    then are still to come when the side stream's kernels run."""
    import torch
    args = inputs()
    want = [t.clone() for t in calls(eg, args, None)]
    n = int(want[3])
    sizes = {t.untyped_storage().nbytes() for t in want}
    sizes |= {eg.engram_embed_grad_workspace_bytes(9000, 2, 64), eg.engram_gate_add_grad_workspace_bytes()}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s if late == "side" else torch.cuda.current_stream()):
            torch.cuda._sleep(20_000_000)
        for size in sizes:
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
        got = calls(eg, args, s if kind == "object" else s.cuda_stream)
        noise = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF) for size in sizes for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        torch.cuda.current_stream().wait_stream(s)
        for i, (a, b) in enumerate(zip(got, want)):
            a, b = (a[:n], b[:n]) if i == 2 else (a, b)
            assert torch.equal(a, b), i
        del got, noise
