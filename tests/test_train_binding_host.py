"""The Python binding of the training calls, without a GPU: what it hands to the library for
tensors of any strides.  Host tensors stand in for device ones (their is_cuda says so); every
call here is refused by the library's argument checks, or goes to a recorder in its place."""
import pytest
import torch


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(t):
    return t.as_subclass(OnDevice)


def zeros(*shape, dtype=torch.float32):
    return dev(torch.zeros(shape, dtype=dtype))


@pytest.fixture(scope="module")
def eg():
    import hashed_gram_memory_gb300 as eg
    return eg


def ids(*shape):
    return zeros(*shape, dtype=torch.int32)


def workspace(eg, *args):
    return zeros(eg.engram_embed_grad_workspace_bytes(*args), dtype=torch.uint8)


def u8(*shape):
    return zeros(*shape, dtype=torch.uint8)


# Views whose rows share elements: broadcast (stride 0) and sliding windows (stride 1).
OVERLAPPING = {
    "broadcast ids": lambda eg: eg.engram_embed(ids(4).expand(100, 4), zeros(9, 16), out=zeros(100, 4, 16), stream=1),
    "one id broadcast": lambda eg: eg.engram_embed(ids(1, 1).expand(100, 1), zeros(9, 16), out=zeros(100, 1, 16),
                                                   stream=1),
    "windows of ids": lambda eg: eg.engram_embed(ids(50).unfold(0, 3, 1), zeros(9, 16), pooled=True, out=zeros(48, 16),
                                                 stream=1),
    "a broadcast table": lambda eg: eg.engram_embed(ids(4, 2), zeros(16).expand(9, 16), out=zeros(4, 2, 16), stream=1),
    "windows as a table": lambda eg: eg.engram_embed(ids(4, 2), zeros(40).unfold(0, 16, 1), out=zeros(4, 2, 16),
                                                     stream=1),
    "gradient, broadcast ids": lambda eg: eg.engram_embed_grad(
        ids(4).expand(100, 4), zeros(100, 4, 8), 9, grad=zeros(9, 8), workspace=workspace(eg, 100, 4, 8), stream=1),
    "gradient, windows of ids": lambda eg: eg.engram_embed_grad_rows(
        ids(50).unfold(0, 3, 1), zeros(48, 3, 8), 9, row_ids=ids(144), grads=zeros(144, 8), count=ids(1),
        workspace=workspace(eg, 48, 3, 8), stream=1),
    "a broadcast gradient buffer": lambda eg: eg.engram_embed_grad(
        ids(5), zeros(5, 8), 9, grad=zeros(8).expand(9, 8), workspace=workspace(eg, 5, 1, 8), stream=1),
    "broadcast gradient rows": lambda eg: eg.engram_embed_grad_rows(
        ids(5), zeros(5, 8), 9, row_ids=ids(5), grads=zeros(8).expand(5, 8), count=ids(1),
        workspace=workspace(eg, 5, 1, 8), stream=1),
    "a broadcast input": lambda eg: eg.engram_fp8_quantise(zeros(256).expand(64, 256), out=[u8(64, 256), u8(64, 2)],
                                                           stream=1),
    "windows as an input": lambda eg: eg.engram_fp8_quantise(
        zeros(300).unfold(0, 256, 1), rows=False, cols=True, out=[eg.fp8_empty(256, 45, "cpu").as_subclass(OnDevice),
                                                                  u8(256, 1)], stream=1),
    "broadcast bytes out": lambda eg: eg.engram_fp8_quantise(zeros(64, 256), out=[u8(256).expand(64, 256), u8(64, 2)],
                                                             stream=1),
    "a broadcast operand": lambda eg: eg.engram_fp8_matmul(u8(128).expand(4, 128), u8(4, 1), u8(8, 128), u8(8, 1),
                                                           out=zeros(4, 8), stream=1),
    "a broadcast product": lambda eg: eg.engram_fp8_matmul(u8(4, 128), u8(4, 1), u8(8, 128), u8(8, 1),
                                                           out=zeros(8).expand(4, 8), stream=1),
}


@pytest.mark.parametrize("what", OVERLAPPING)
def test_rows_that_share_elements_are_refused(eg, what):
    """The library reads and writes rows that are at least their width apart; a view with less
    is refused, not read with another stride than its own."""
    with pytest.raises(eg.EngramError) as e:
        OVERLAPPING[what](eg)
    assert e.value.code == eg.ERR_INVALID_ARG, str(e.value)


class Recorder:
    """Takes the library's place: keeps each call's arguments and reports success."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def recorder(eg, monkeypatch):
    r = Recorder(eg.lib)
    monkeypatch.setattr(eg, "lib", r)
    return r


def test_strides_of_rows_go_through(eg, recorder):
    """Padded rows, and a single row, whose stride says nothing."""
    eg.engram_embed(ids(10, 12)[:, 4:8], zeros(9, 24)[:, :16], out=zeros(10, 4, 16), stream=1)
    eg.engram_embed(ids(4).expand(1, 4), zeros(16).expand(1, 16), out=zeros(1, 4, 16), stream=1)
    eg.engram_embed(ids(1, 10).t(), zeros(9, 16), out=zeros(10, 1, 16), stream=1)
    for (_, a), want in zip(recorder.calls, [(4, 12, 24), (4, 4, 16), (1, 1, 16)]):
        assert (a[2], a[3], a[8]) == want
    recorder.calls.clear()
    for x, stride in ((zeros(6, 48)[:, :32], 48), (zeros(6, 48)[3:4, :32], 48), (zeros(32).expand(1, 32), 32),
                      (zeros(1, 6).t(), 1)):
        M, K = x.shape
        eg.engram_fp8_quantise(x, out=[u8(M, 32)[:, :K], u8(M, 1)], stream=1)
        assert recorder.calls.pop()[1][4] == stride
    for out, stride in ((zeros(4, 12)[:, :8], 12), (zeros(4, 8), 8)):
        eg.engram_fp8_matmul(u8(4, 128), u8(4, 1), u8(8, 128), u8(8, 1), out=out, stream=1)
        assert recorder.calls.pop()[1][13] == stride
    eg.engram_embed_grad(ids(5), zeros(5, 8), 9, grad=zeros(9, 12)[:, :8], workspace=workspace(eg, 5, 1, 8), stream=1)
    assert recorder.calls.pop()[1][14] == 12


# Scratch that is not a run of device bytes: host memory, and views that hold less than they say.
SCRATCH = {"host memory": lambda n: torch.zeros(n, dtype=torch.uint8), "a broadcast byte": lambda n: u8(1).expand(n),
           "every other byte": lambda n: u8(2 * n)[::2]}


@pytest.mark.parametrize("kind", SCRATCH)
def test_scratch_must_be_device_memory_in_one_piece(eg, recorder, kind):
    def scratch(n):
        return SCRATCH[kind](n)
    n = eg.engram_embed_grad_workspace_bytes(5, 1, 8)
    for call in (lambda: eg.engram_embed_grad(ids(5), zeros(5, 8), 9, grad=zeros(9, 8), workspace=scratch(n), stream=1),
                 lambda: eg.engram_embed_grad_rows(ids(5), zeros(5, 8), 9, row_ids=ids(5), grads=zeros(5, 8),
                                                   count=ids(1), workspace=scratch(n), stream=1),
                 lambda: eg.engram_gate_add_grad(zeros(3, 16), None, zeros(3, 4, 16, dtype=torch.bfloat16), zeros(4),
                                                 zeros(3, 4, 16, dtype=torch.bfloat16),
                                                 dx=zeros(3, 4, 16, dtype=torch.bfloat16), dk=zeros(3, 16),
                                                 dalpha=zeros(4), stream=1,
                                                 workspace=scratch(eg.engram_gate_add_grad_workspace_bytes()))):
        with pytest.raises(eg.EngramError) as e:
            call()
        assert e.value.code == eg.ERR_INVALID_ARG and "workspace" in str(e.value)
    assert recorder.calls == []
