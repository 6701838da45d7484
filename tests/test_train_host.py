"""The training calls on the host, without a GPU: every argument error comes back before
anything touches a device, and the workspace queries answer."""
import ctypes as C

import pytest

P, Q, S, W, O = (i << 24 for i in range(1, 6))  # far apart, 16-byte aligned
BF16, F32 = 0, 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def eg():
    import hashed_gram_memory_gb300 as eg
    return eg


def refuses(eg, name, base, changes, code=None):
    f = getattr(eg.lib, name)
    names = list(base)
    for change in changes:
        args = dict(base, **change)
        got = f(*[args[n] for n in names])
        assert got == (code or eg.ERR_INVALID_ARG), (name, change, got)
        assert eg.lib.engram_last_error().decode().startswith(name), change


def test_embed_argument_errors(eg):
    base = dict(ids=P, n=10, r=4, ids_stride=4, table=Q, td=BF16, rows=100, D=32, ts=32, scale=1.0,
                pooled=0, out=O, od=BF16, tok=128, per=32, status=None, stream=None)
    refuses(eg, "engram_embed", base, [
        dict(ids=None), dict(ids=P + 2), dict(n=-1), dict(r=0), dict(n=2 ** 30), dict(ids_stride=3),
        dict(table=None), dict(table=Q + 1), dict(td=2), dict(td=-1), dict(rows=0), dict(rows=2 ** 31),
        dict(D=0), dict(D=16385), dict(ts=31), dict(out=None), dict(out=O + 1), dict(od=7), dict(tok=127),
        dict(per=31), dict(pooled=1, tok=31), dict(status=W + 2), dict(out=P), dict(out=Q),
        dict(out=O, status=O), dict(td=F32, table=Q + 2)])
    assert eg.lib.engram_embed(None, 0, 4, 4, Q, 0, 100, 32, 32, 1.0, 0, None, 0, 128, 32, None, None) == eg.OK


def test_embed_grad_argument_errors(eg):
    need = eg.engram_embed_grad_workspace_bytes(10, 4, 32)
    assert need > 0
    base = dict(ids=P, n=10, r=4, ids_stride=4, dy=Q, dd=BF16, tok=128, per=32, rows=100, D=32, scale=1.0,
                acc=0, grad=O, gd=F32, gs=32, ws=W, wb=need, status=None, stream=None)
    common = [dict(ids=None), dict(ids=P + 1), dict(n=-1), dict(r=0), dict(n=2 ** 30), dict(ids_stride=3),
              dict(dy=None), dict(dy=Q + 1), dict(dd=3), dict(tok=-1), dict(per=-1), dict(rows=0),
              dict(rows=2 ** 31), dict(D=0), dict(D=16385), dict(ws=None), dict(ws=W + 8), dict(wb=need - 1),
              dict(status=S + 2), dict(ws=P)]
    refuses(eg, "engram_embed_grad", base, common + [
        dict(grad=None), dict(grad=O + 2), dict(gd=9), dict(gs=31), dict(grad=Q), dict(grad=W), dict(grad=P)])
    rows = dict(ids=P, n=10, r=4, ids_stride=4, dy=Q, dd=BF16, tok=128, per=32, rows=100, D=32, scale=1.0,
                row_ids=S, grads=O, gd=F32, gs=32, count=S + 4096, ws=W, wb=need, status=None, stream=None)
    refuses(eg, "engram_embed_grad_rows", rows, [c for c in common if "status" not in c] + [
        dict(grads=None), dict(gs=31), dict(row_ids=None), dict(row_ids=S + 1), dict(count=None),
        dict(count=S), dict(grads=S), dict(row_ids=P), dict(count=Q)])


def test_workspace_queries(eg):
    f = eg.engram_embed_grad_workspace_bytes
    assert f(-1, 1, 8) == 0 and f(1, 0, 8) == 0 and f(1, 1, 0) == 0 and f(2 ** 31, 1, 8) == 0
    assert f(0, 1, 8) > 0
    # two lists of pairs, and little beside them for narrow rows
    assert 16 * 65536 * 24 <= f(65536, 24, 8) <= 32 * 65536 * 24
    assert f(4096, 1, 4096) >= f(4096, 1, 64)
    assert eg.engram_gate_add_grad_workspace_bytes() >= 16 * 304


def test_quantise_argument_errors(eg):
    base = dict(x=P, xd=F32, M=10, K=200, xs=200, br=1, q=Q, qs=208, s=S, qt=O, qts=16, st=W, status=None,
                stream=None)
    refuses(eg, "engram_fp8_quantise", base, [
        dict(x=None), dict(x=P + 2), dict(xd=5), dict(M=-1), dict(K=0), dict(xs=199), dict(br=0), dict(br=64),
        dict(q=None, qt=None), dict(s=None), dict(st=None), dict(q=Q + 8), dict(qt=O + 1), dict(qs=200),
        dict(qs=192), dict(qts=8), dict(q=P), dict(qt=P), dict(qt=Q), dict(st=S), dict(s=P), dict(status=Q),
        dict(status=W + 4097)])
    refuses(eg, "engram_fp8_quantise", dict(base, M=2 ** 31 - 1, K=2 ** 31 - 1, xs=2 ** 31), [dict()],
            eg.ERR_UNSUPPORTED)
    args = dict(base, M=0, x=None, q=None, s=None, qt=None, st=None)
    assert eg.lib.engram_fp8_quantise(*args.values()) == eg.OK


def test_matmul_argument_errors(eg):
    base = dict(a=P, sa=208, a_scale=S, ab=1, b=Q, sb=208, b_scale=S + 65536, bb=128, M=10, N=20, K=200, out=O,
                od=F32, so=20, status=None, stream=None)
    refuses(eg, "engram_fp8_matmul", base, [
        dict(a=None), dict(b=None), dict(a_scale=None), dict(b_scale=None), dict(out=None), dict(a=P + 8),
        dict(b=Q + 4), dict(sa=200), dict(sa=192), dict(sb=204), dict(sb=0), dict(ab=2), dict(bb=0), dict(M=-1),
        dict(N=-1), dict(K=0), dict(K=2 ** 31), dict(od=2), dict(out=O + 2), dict(so=19), dict(status=W + 1),
        dict(out=P), dict(out=Q), dict(out=S), dict(out=S + 65536), dict(status=O)])
    for empty in (dict(M=0), dict(N=0)):
        assert eg.lib.engram_fp8_matmul(*dict(base, a=None, b=None, out=None, **empty).values()) == eg.OK


def test_gate_grad_argument_errors(eg):
    need = eg.engram_gate_add_grad_workspace_bytes()
    base = dict(k=P, state=None, n=10, D=64, x=Q, alpha=W, eps=1e-6, dy=S, dx=O, dk=O + (1 << 20), kd=F32,
                dalpha=W + 64, ws=W + 4096, wb=need, stream=None)
    refuses(eg, "engram_gate_add_grad", base, [
        dict(k=None), dict(k=P + 4), dict(n=-1), dict(n=2 ** 31), dict(D=8), dict(D=24), dict(D=8208), dict(x=None),
        dict(x=Q + 2), dict(alpha=None), dict(alpha=W + 1), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
        dict(dy=None), dict(dx=None), dict(dk=None), dict(dk=O + (1 << 20) + 8), dict(kd=4), dict(dalpha=None),
        dict(dalpha=W + 65), dict(ws=None), dict(ws=W + 4104), dict(wb=need - 1), dict(dx=Q), dict(dx=S + 512),
        dict(dk=P), dict(dalpha=W + 8), dict(dk=O), dict(ws=W + 64)])


def test_binding_rejects_cpu_tensors(eg):
    import torch
    ids, t = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, 16)
    q, s = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    for call in (lambda: eg.engram_embed(ids, t), lambda: eg.engram_embed_grad(ids, torch.zeros(4, 2, 16), 8),
                 lambda: eg.engram_embed_grad_rows(ids, torch.zeros(4, 2, 16), 8),
                 lambda: eg.engram_fp8_quantise(t), lambda: eg.engram_fp8_matmul(q, s, q, s),
                 lambda: eg.engram_gate_add_grad(t, None, torch.zeros(8, 4, 16), torch.zeros(4),
                                                 torch.zeros(8, 4, 16))):
        with pytest.raises(eg.EngramError) as e:
            call()
        assert e.value.code == eg.ERR_INVALID_ARG and "CUDA" in str(e.value)


def test_training_dtypes_match_the_header(eg):
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "engram.h")).read()
    want = {k: int(v) for k, v in re.findall(r"#define ENGRAM_(DTYPE_\w+|MAX_EMBED_D|FP8_BLOCK) (\d+)", src)}
    assert want == {"DTYPE_BF16": eg.DTYPE_BF16, "DTYPE_F32": eg.DTYPE_F32, "MAX_EMBED_D": eg.MAX_EMBED_D,
                    "FP8_BLOCK": eg.FP8_BLOCK}
    assert C.sizeof(C.c_int32) == 4
