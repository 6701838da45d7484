"""Memory that the Python binding makes for a call, without a GPU: it has to belong to the stream
that the call launches on.  Scratch of another stream's pool could be handed out again while the
kernels still use it, and a result could start in memory that the other stream still works on."""
import contextlib

import pytest
import torch

CURRENT, SIDE = 11, 22  # raw stream handles


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Library:
    """Takes the library's place: reports success, keeps the calls' names and streams."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args[-1]))
            return 0
        return call


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def world(monkeypatch):
    """The binding over host tensors: which stream each allocation is made under, and which
    streams its tensors are recorded on."""
    import hashed_gram_memory_gb300 as eg
    state = {"now": CURRENT, "made": [], "recorded": []}

    @contextlib.contextmanager
    def under(stream):
        before, state["now"] = state["now"], stream.cuda_stream
        yield
        state["now"] = before

    def maker(real):
        def make(*args, **kw):
            state["made"].append(state["now"])
            return real(*args, **kw).as_subclass(OnDevice)
        return make
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(state["now"]))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: state["now"], raising=False)
    monkeypatch.setattr(OnDevice, "record_stream", lambda t, s: state["recorded"].append(s.cuda_stream), raising=False)
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, maker(getattr(torch, name)))
    monkeypatch.setattr(eg, "lib", Library(eg.lib))
    return eg, state


def i32(*shape):
    return zeros(*shape, dtype=torch.int32)


def u8(*shape):
    return zeros(*shape, dtype=torch.uint8)


def bf(*shape):
    return zeros(*shape, dtype=torch.bfloat16)


def tables(eg):
    return eg.Tables(eg.TABLE_BF16, [bf(7, 32) for _ in range(3)])


# call: (how it is called, results it makes, scratch buffers it makes)
CALLS = {
    "embed": (lambda eg, s: eg.engram_embed(i32(5, 2), zeros(9, 16), stream=s), 1, 0),
    "embed_grad": (lambda eg, s: eg.engram_embed_grad(i32(5, 2), zeros(5, 2, 16), 9, stream=s), 1, 1),
    "embed_grad_rows": (lambda eg, s: eg.engram_embed_grad_rows(i32(5, 2), zeros(5, 2, 16), 9, stream=s), 3, 1),
    "quantise": (lambda eg, s: eg.engram_fp8_quantise(zeros(5, 200), cols=True, stream=s), 4, 0),
    "matmul": (lambda eg, s: eg.engram_fp8_matmul(u8(4, 128), u8(4, 1), u8(8, 128), u8(8, 1), stream=s), 1, 0),
    "gate_add_grad": (lambda eg, s: eg.engram_gate_add_grad(zeros(3, 16), None, bf(3, 4, 16), zeros(4), bf(3, 4, 16),
                                                            stream=s), 3, 1),
    "pack_e8m0_rows": (lambda eg, s: eg.engram_pack_e8m0_rows(u8(4, 64), u8(4, 2), stream=s), 1, 0),
    "compress": (lambda eg, s: eg.engram_compress(i32(2, 3), i32(9), 9, stream=s), 1, 0),
    "hash": (lambda eg, s: eg.engram_hash(i32(2, 3), 2, (7, 7, 7), stream=s), 1, 0),
    "compress_hash": (lambda eg, s: eg.engram_compress_hash(i32(2, 3), i32(9), 9, 2, (7, 7, 7), stream=s), 1, 0),
    "lookup_fused": (lambda eg, s: eg.engram_lookup_fused(i32(2, 3, 2), 2, tables(eg), bf(2, 4, 32), zeros(4),
                                                          stream=s), 1, 0),
    "concat_rows": (lambda eg, s: eg.engram_concat_rows(i32(2, 3, 2), 2, tables(eg), stream=s), 2, 0),
    "wkv_project": (lambda eg, s: eg.engram_wkv_project(bf(2, 64), bf(32, 64), stream=s), 1, 0),
    "gate_add": (lambda eg, s: eg.engram_gate_add(zeros(2, 32), u8(2), bf(2, 4, 32), zeros(4), stream=s), 1, 0),
    "connection": (lambda eg, s: eg.engram_connection(i32(2, 3, 2), 2, tables(eg), bf(64, 192), bf(2, 4, 64), zeros(4),
                                                      stream=s), 1, 1),
    "forward": (lambda eg, s: eg.engram_forward(i32(1, 2), i32(9), 9, 2, tables(eg), bf(2, 4, 32), zeros(4),
                                                stream=s), 1, 1),
    "forward_static": (lambda eg, s: eg.engram_forward_static(i32(1, 2), i32(9), 9, 2, tables(eg), bf(2, 4, 32),
                                                              zeros(4), stream=s), 1, 0),
}


@pytest.mark.parametrize("kind", ["handle", "object"])
@pytest.mark.parametrize("name", CALLS)
def test_a_side_streams_call_allocates_on_it(world, name, kind):
    eg, state = world
    call, results, scratch = CALLS[name]
    call(eg, SIDE if kind == "handle" else Stream(SIDE))
    assert state["made"] == [SIDE] * (results + scratch)
    assert state["now"] == CURRENT
    # the caller reads the results from the current stream: they outlive its work too
    assert state["recorded"] == [CURRENT] * results
    assert len(eg.lib.calls) == 1 and eg.lib.calls[0][1] == SIDE


@pytest.mark.parametrize("stream", [None, CURRENT, Stream(CURRENT)], ids=["none", "handle", "object"])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_streams_call_allocates_plainly(world, name, stream):
    eg, state = world
    call, results, scratch = CALLS[name]
    call(eg, stream)
    assert state["made"] == [CURRENT] * (results + scratch) and state["recorded"] == []
    assert eg.lib.calls[0][1] == CURRENT


def test_the_default_stream_by_its_handle(world, monkeypatch):
    """0 is the default stream, which torch does not take as an external one."""
    eg, state = world
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    CALLS["embed_grad"][0](eg, 0)
    assert state["made"] == [0, 0] and eg.lib.calls[0][1] == 0
