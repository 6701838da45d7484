"""engram_matmul, engram_matmul_grad and engram_orthogonalise on the host, without a GPU: every
argument error comes back before anything touches a device, the workspace queries answer, and the
binding hands tensors of any strides to the library as they are.  Host tensors stand in for device
ones (their is_cuda says so)."""
import struct

import pytest
import torch

A, B, O, R, Z, W, V, S = (i << 24 for i in range(1, 9))  # far apart, 16-byte aligned
BF16, F32 = 0, 1
NAN, INF = float("nan"), float("inf")
MATMUL = ("a", "a_stride", "b", "b_stride", "M", "N", "K", "bias", "residual", "residual_stride", "pre", "pre_stride",
          "out", "out_stride", "a_trans", "b_trans", "activation", "bias_dtype", "residual_dtype", "pre_dtype",
          "out_dtype", "scale")
GRAD = ("dy", "dy_stride", "a", "a_stride", "b", "b_stride", "M", "N", "K", "pre", "pre_stride", "da", "da_stride",
        "db", "db_stride", "dbias", "a_trans", "b_trans", "activation", "dy_dtype", "pre_dtype", "da_dtype",
        "db_dtype", "accumulate", "scale")


@pytest.fixture(scope="module")
def eg():
    import hashed_gram_memory_gb300 as eg
    return eg


def packed(eg, names, values):
    fmt = eg._MATMUL_ARGS if names is MATMUL else eg._MATMUL_GRAD_ARGS
    return fmt.pack(*(values[n] for n in names))


def matmul(eg, **change):
    v = dict(a=A, a_stride=64, b=B, b_stride=64, M=10, N=40, K=64, bias=0, residual=0, residual_stride=0, pre=0,
             pre_stride=0, out=O, out_stride=40, a_trans=0, b_trans=0, activation=0, bias_dtype=F32,
             residual_dtype=F32, pre_dtype=F32, out_dtype=F32, scale=1.0, ws=None, ws_bytes=0, status=None)
    v.update(change)
    return eg.lib.engram_matmul(packed(eg, MATMUL, v), v["ws"], v["ws_bytes"], v["status"], None)


def grad(eg, **change):
    v = dict(dy=Z, dy_stride=40, a=A, a_stride=64, b=B, b_stride=64, M=10, N=40, K=64, pre=0, pre_stride=0, da=O,
             da_stride=64, db=R, db_stride=64, dbias=V, a_trans=0, b_trans=0, activation=0, dy_dtype=BF16,
             pre_dtype=BF16, da_dtype=BF16, db_dtype=F32, accumulate=0, scale=1.0, ws=W, ws_bytes=1 << 20, status=None)
    v.update(change)
    return eg.lib.engram_matmul_grad(packed(eg, GRAD, v), v["ws"], v["ws_bytes"], v["status"], None)


def orth(eg, **change):
    v = dict(g=A, gd=F32, L=2, M=10, N=40, gb=400, gs=40, mom=B, mb=400, ms=40, beta=0.9, nesterov=1, steps=5, a=3.4,
             b=-4.8, c=2.0, scale=1.0, eps=1e-7, out=O, ob=400, os=40, ws=W, wb=None, status=None, stream=None)
    v.update(change)
    if v["wb"] is None:
        v["wb"] = max(eg.lib.engram_orthogonalise_workspace_bytes(v["L"], v["M"], v["N"]), 1 << 16)
    return eg.lib.engram_orthogonalise(*v.values())


MATMUL_ERRORS = [
    dict(a=0), dict(a=A + 1), dict(a_stride=63), dict(b=0), dict(b=B + 1), dict(b_stride=-64), dict(out=0),
    dict(out=O + 2), dict(out_stride=39), dict(M=-1), dict(N=0), dict(K=0), dict(M=2 ** 31 - 256), dict(N=2 ** 31),
    dict(K=2 ** 33), dict(activation=4), dict(activation=-1), dict(out_dtype=2), dict(bias=V + 2),
    dict(bias=V, bias_dtype=3), dict(residual=R, residual_dtype=-1), dict(residual=R, residual_stride=-1),
    dict(residual=R + 2, residual_stride=40), dict(pre=Z, pre_stride=39), dict(pre=Z + 1, pre_stride=40, pre_dtype=BF16),
    dict(pre=Z, pre_stride=40, pre_dtype=7), dict(status=S + 2), dict(a_trans=1, a_stride=9), dict(b_trans=1, b_stride=39),
    dict(a_stride=2 ** 39), dict(out_stride=2 ** 39),
    # rows off 16-byte boundaries need a workspace
    dict(a_stride=65), dict(a=A + 2), dict(b_trans=1, b_stride=41), dict(a=A + 8, ws=W, ws_bytes=1),
    dict(a=A + 8, ws=W + 8, ws_bytes=1 << 20),
    # overlapping buffers
    dict(out=A), dict(out=B), dict(pre=O, pre_stride=40), dict(pre=A, pre_stride=40), dict(bias=O),
    dict(residual=O, residual_stride=41), dict(residual=O, residual_stride=40, residual_dtype=BF16),
    dict(residual=O + 160, residual_stride=40), dict(status=O), dict(a=A + 2, ws=A, ws_bytes=1 << 20),
    dict(a=A + 2, ws=O, ws_bytes=1 << 20)]


@pytest.mark.parametrize("i", range(len(MATMUL_ERRORS)))
def test_matmul_argument_errors(eg, i):
    assert matmul(eg, **MATMUL_ERRORS[i]) == eg.ERR_INVALID_ARG, MATMUL_ERRORS[i]
    assert eg.lib.engram_last_error().decode().startswith("engram_matmul: ")


GRAD_ERRORS = [
    dict(dy=0), dict(dy=Z + 1), dict(dy_stride=-40), dict(dy_dtype=4), dict(a=0), dict(b=0), dict(b=B + 1),
    dict(a_stride=10), dict(M=-1), dict(N=0), dict(K=0), dict(M=2 ** 31), dict(activation=9), dict(activation=2),
    dict(activation=1, pre=S, pre_dtype=4, pre_stride=40), dict(activation=1, pre=S + 1, pre_stride=40),
    dict(activation=3, pre=S, pre_stride=-1), dict(da=0, db=0, dbias=0), dict(da_dtype=2), dict(db_dtype=-1),
    dict(da_stride=63), dict(db_stride=63), dict(da=O + 1), dict(db=R + 2), dict(dbias=V + 2), dict(status=S + 1),
    dict(activation=1, pre=S, pre_stride=40, ws=None), dict(dy_dtype=F32, ws_bytes=100), dict(a=A + 2, ws_bytes=64),
    dict(dy=Z + 2, ws=W + 4),
    dict(da=Z), dict(db=A), dict(da=B), dict(dbias=Z), dict(db=O), dict(dbias=O), dict(dy_dtype=F32, ws=Z),
    dict(dy_dtype=F32, ws=O), dict(activation=1, pre=R, pre_stride=40), dict(status=V)]


@pytest.mark.parametrize("i", range(len(GRAD_ERRORS)))
def test_gradient_argument_errors(eg, i):
    assert grad(eg, **GRAD_ERRORS[i]) == eg.ERR_INVALID_ARG, GRAD_ERRORS[i]
    assert eg.lib.engram_last_error().decode().startswith("engram_matmul_grad: ")


ORTH_ERRORS = [
    dict(g=0), dict(g=A + 2), dict(gd=2), dict(L=-1), dict(L=65536), dict(M=0), dict(N=0), dict(M=2 ** 31), dict(gs=39),
    dict(gb=399), dict(mom=B + 2), dict(ms=39), dict(mb=399), dict(out=0), dict(out=O + 1), dict(os=39), dict(ob=399),
    dict(steps=0), dict(steps=65), dict(a=17.0), dict(b=NAN), dict(c=-INF), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN),
    dict(scale=INF), dict(beta=NAN), dict(ws=None), dict(ws=W + 8), dict(wb=100), dict(status=S + 2), dict(out=A),
    dict(mom=A), dict(out=B), dict(ws=A), dict(ws=O), dict(status=O), dict(gs=2 ** 39)]


@pytest.mark.parametrize("i", range(len(ORTH_ERRORS)))
def test_orthogonalise_argument_errors(eg, i):
    assert orth(eg, **ORTH_ERRORS[i]) == eg.ERR_INVALID_ARG, ORTH_ERRORS[i]
    assert eg.lib.engram_last_error().decode().startswith("engram_orthogonalise: ")


def test_nothing_to_do(eg):
    assert eg.lib.engram_matmul(None, None, 0, None, None) == eg.ERR_INVALID_ARG
    assert eg.lib.engram_matmul_grad(None, None, 0, None, None) == eg.ERR_INVALID_ARG
    assert matmul(eg, M=0, a=0, out=0) == eg.OK
    assert orth(eg, L=0, g=0, out=0, ws=None) == eg.OK


def test_workspace_queries(eg):
    def m(**change):
        v = dict.fromkeys(MATMUL, 0) | dict(a=A, a_stride=64, b=B, b_stride=64, M=10, N=40, K=64, scale=1.0) | change
        return eg.lib.engram_matmul_workspace_bytes(packed(eg, MATMUL, v))
    assert m() == 0 and m(M=1, a_stride=3) == 0 and m(a_trans=1, a_stride=16) == 0
    assert m(a=A + 2) >= 10 * 64 * 2 and m(a_stride=65) >= 10 * 64 * 2 and m(b_stride=66) >= 40 * 64 * 2
    assert m(a_trans=1, a_stride=10) >= 64 * 16 * 2 and m(N=0) == 0
    assert eg.lib.engram_matmul_workspace_bytes(None) == 0

    def g(**change):
        v = dict.fromkeys(GRAD, 0) | dict(dy=Z, dy_stride=64, a=A, a_stride=64, b=B, b_stride=64, M=2000, N=64, K=64,
                                          da=O, db=R, scale=1.0) | change
        return eg.lib.engram_matmul_grad_workspace_bytes(packed(eg, GRAD, v))
    assert g() == 0 and g(M=0) == 0
    assert g(dy_dtype=F32) >= 2000 * 64 * 2 and g(activation=1) >= 2000 * 64 * 2 and g(dy_stride=0) >= 2000 * 64 * 2
    assert 0 < g(dbias=V) < 2000 * 64 * 2 and g(dbias=V, M=500) == 0 and g(dy_dtype=F32, da=0, db=0) == 0
    f = eg.engram_orthogonalise_workspace_bytes
    assert f(1, 0, 4) == 0 and f(-1, 4, 4) == 0 and f(3, 100, 200) >= 3 * 2 * (2 * 100 * 200 + 2 * 100 * 100)


# ------------------------------------------------------------------------ the binding

class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def bf(*shape):
    return zeros(*shape, dtype=torch.bfloat16)


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


def last(eg, recorder, names):
    name, args = recorder.calls.pop()
    fmt = eg._MATMUL_ARGS if names is MATMUL else eg._MATMUL_GRAD_ARGS
    return dict(zip(names, fmt.unpack(args[0])))


def test_strides_and_layouts_go_through(eg, recorder):
    a, w = bf(10, 80)[:, 8:72], bf(64, 40)
    out, pre = zeros(10, 48)[:, :40], zeros(10, 40, dtype=torch.bfloat16)
    eg.engram_matmul(a, w.t(), bias=zeros(40), residual=zeros(40).expand(10, 40), activation=eg.ACT_SILU, scale=0.5,
                     pre=pre, out=out, stream=1)
    v = last(eg, recorder, MATMUL)
    assert (v["a"], v["a_stride"], v["a_trans"]) == (a.data_ptr(), 80, 0)
    assert (v["b"], v["b_stride"], v["b_trans"]) == (w.data_ptr(), 40, 1)
    assert (v["M"], v["N"], v["K"], v["activation"], v["scale"]) == (10, 40, 64, 2, 0.5)
    assert (v["residual_stride"], v["pre_stride"], v["out_stride"]) == (0, 40, 48)
    assert (v["bias_dtype"], v["residual_dtype"], v["pre_dtype"], v["out_dtype"]) == (1, 1, 0, 1)
    eg.engram_matmul(bf(1, 64), bf(64, 9)[:, :1].t(), out=zeros(1, 1), stream=1,
                     workspace=zeros(4096, dtype=torch.uint8))  # one row: a column of memory
    v = last(eg, recorder, MATMUL)
    assert (v["b_stride"], v["b_trans"]) == (9, 1)
    eg.engram_matmul_grad(zeros(10, 40), a, w.t(), da=bf(10, 70)[:, :64], db=zeros(40, 64), dbias=zeros(40),
                          grad_bias=True, accumulate=True, workspace=zeros(1 << 16, dtype=torch.uint8), stream=1)
    v = last(eg, recorder, GRAD)
    assert (v["dy_dtype"], v["da_stride"], v["db_dtype"], v["accumulate"], v["pre"]) == (1, 70, 1, 1, 0)
    g = bf(3, 12, 50)[:, 1:11, :40]
    eg.engram_orthogonalise(g, momentum=zeros(3, 10, 40), out=bf(3, 10, 40), stream=1,
                            workspace=zeros(1 << 16, dtype=torch.uint8))
    name, args = recorder.calls.pop()
    assert args[1:7] == (0, 3, 10, 40, 600, 50) and args[8:10] == (400, 40)


REFUSED = {
    "K disagrees": lambda e: e.engram_matmul(bf(4, 8), bf(5, 16), out=zeros(4, 5), stream=1),
    "three dimensions": lambda e: e.engram_matmul(bf(1, 4, 8), bf(5, 8), out=zeros(4, 5), stream=1),
    "no dense dimension": lambda e: e.engram_matmul(bf(8, 32)[::2, ::2], bf(5, 16), out=zeros(4, 5), stream=1),
    "fp32 operand": lambda e: e.engram_matmul(zeros(4, 8), bf(5, 8), out=zeros(4, 5), stream=1),
    "host operand": lambda e: e.engram_matmul(torch.zeros(4, 8, dtype=torch.bfloat16), bf(5, 8), out=zeros(4, 5), stream=1),
    "bias size": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), bias=zeros(4), out=zeros(4, 5), stream=1),
    "bias strides": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), bias=zeros(10)[::2], out=zeros(4, 5), stream=1),
    "out size": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), out=zeros(5, 4), stream=1),
    "out columns": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), out=zeros(5, 4).t(), stream=1),
    "broadcast out": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), out=zeros(5).expand(4, 5), stream=1),
    "broadcast operand": lambda e: e.engram_matmul(bf(8).expand(4, 8), bf(5, 8), out=zeros(4, 5), stream=1),
    "residual size": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), residual=zeros(5), out=zeros(4, 5), stream=1),
    "pre type": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), pre=zeros(4, 5, dtype=torch.float64), out=zeros(4, 5), stream=1),
    "activation": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), activation=7, out=zeros(4, 5), stream=1),
    "activation by name": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), activation="relu", out=zeros(4, 5), stream=1),
    "host workspace": lambda e: e.engram_matmul(bf(4, 9), bf(5, 9), out=zeros(4, 5), stream=1,
                                                workspace=torch.zeros(4096, dtype=torch.uint8)),
    "dy size": lambda e: e.engram_matmul_grad(bf(4, 6), bf(4, 8), bf(5, 8), stream=1),
    "no pre": lambda e: e.engram_matmul_grad(bf(4, 5), bf(4, 8), bf(5, 8), activation=1, stream=1),
    "nothing to add to": lambda e: e.engram_matmul_grad(bf(4, 5), bf(4, 8), bf(5, 8), accumulate=True, stream=1),
    "dbias type": lambda e: e.engram_matmul_grad(bf(4, 5), bf(4, 8), bf(5, 8), da=bf(4, 8), db=bf(5, 8), grad_bias=True,
                                                 dbias=bf(5), stream=1),
    "nothing asked for": lambda e: e.engram_matmul_grad(bf(4, 8), bf(4, 8), bf(8, 8), grad_a=False, grad_b=False, stream=1),
    "one dimension": lambda e: e.engram_orthogonalise(zeros(8), out=bf(8), stream=1),
    "bf16 momentum": lambda e: e.engram_orthogonalise(zeros(8, 8), momentum=bf(8, 8), out=bf(8, 8), stream=1),
    "momentum size": lambda e: e.engram_orthogonalise(zeros(8, 8), momentum=zeros(8, 9), out=bf(8, 8), stream=1,
                                                      workspace=zeros(1 << 16, dtype=torch.uint8)),
    "fp32 out": lambda e: e.engram_orthogonalise(zeros(8, 8), out=zeros(8, 8), stream=1),
    "two coefficients": lambda e: e.engram_orthogonalise(zeros(8, 8), coefficients=(1.5, -0.5), out=bf(8, 8), stream=1),
    "transposed gradient": lambda e: e.engram_orthogonalise(zeros(8, 9).t(), out=bf(9, 8), stream=1,
                                                            workspace=zeros(1 << 16, dtype=torch.uint8)),
    "matrices that overlap": lambda e: e.engram_orthogonalise(zeros(8, 9).expand(3, 8, 9), out=bf(3, 8, 9), stream=1,
                                                              workspace=zeros(1 << 16, dtype=torch.uint8)),
}


@pytest.mark.parametrize("what", REFUSED)
def test_binding_refusals(eg, what):
    with pytest.raises(eg.EngramError) as e:
        REFUSED[what](eg)
    assert e.value.code == eg.ERR_INVALID_ARG, str(e.value)


def test_tensors_on_two_devices_are_refused(eg, recorder):
    class Elsewhere(OnDevice):
        def get_device(self):
            return 1
    with pytest.raises(eg.EngramError, match="one device"):
        eg.engram_matmul(bf(4, 8), bf(5, 8).as_subclass(Elsewhere), out=zeros(4, 5), stream=1)
    with pytest.raises(eg.EngramError, match="one device"):
        eg.engram_orthogonalise(zeros(8, 8), out=bf(8, 8).as_subclass(Elsewhere), stream=1,
                                workspace=zeros(1 << 16, dtype=torch.uint8))
    assert recorder.calls == []


def test_argument_structs_have_the_headers_layout(eg):
    """Pointers and 64-bit numbers first, then 32-bit ones: no gaps but at the end."""
    assert eg._MATMUL_ARGS.size == 14 * 8 + 8 * 4 and eg._MATMUL_GRAD_ARGS.size == 16 * 8 + 9 * 4 + 4
    assert struct.calcsize("P") == 8
