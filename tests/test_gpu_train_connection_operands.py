"""The training example's two passes link by link, in fp64 on the very operands that its 8-bit
products read: the quantised copies' values, the kernels' own k, dk and dE.  Each link's
tolerance is that of its operator's own test (test_gpu_fp8.py, test_gpu_gate_grad.py,
test_gpu_embed_grad.py), so a swapped copy, a wrong scale or a missing term of a few
thousandths shows, which a comparison with the unquantised chain cannot see."""
import importlib.util
import os

import numpy as np
import pytest

from tests import test_gpu_embed_grad as rows_test, test_gpu_fp8 as fp8_test, test_gpu_gate_grad as gate_test

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location(
        "train_connection_links", os.path.join(ROOT, "examples", "train_connection.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def quantised(x, block_rows=1):
    """The fp64 values that x [M, K] has once quantised along K, from the definition."""
    q, s = fp8_test.reference(x.double().cpu().numpy(), block_rows)
    wide = np.exp2(s.astype(np.float64) - 127).repeat(128, 1)[:, :x.shape[1]]
    return fp8_test.VALUES[q] * wide.repeat(block_rows, 0)[:x.shape[0]]


def test_every_link_in_fp64(example):
    import torch
    eg = example.eg
    net = example.Connection(seed=4)
    T = 333
    g = torch.Generator(device="cuda").manual_seed(6)
    tokens = torch.randint(0, net.n_eids, (1, T), generator=g, device="cuda", dtype=torch.int32)
    dead = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    dead[0, ::9] = 1
    x = torch.randn(T, 4, net.hidden, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, 4, net.hidden, generator=g, device="cuda").bfloat16()
    ids = net.row_ids(tokens, dead)
    y, saved = net.forward(ids, x)
    k, state = saved[2], saved[3]
    dx, dalpha, dwkv, (row_ids, grads, count) = net.backward(saved, dy)
    assert eg.engram_read_status(net.status) == (eg.OK, 0)

    live = state == 0
    assert torch.equal(live, ids[:, 0] >= 0) and 0 < int(live.sum()) < T
    e = (net.table[ids.long().clamp(min=0)] * (ids >= 0).unsqueeze(-1)).reshape(T, net.K)
    fp8_test.check_product(k, quantised(e), quantised(net.wkv, 128), False)

    dx2, dk, dalpha2 = eg.engram_gate_add_grad(k, state, x, net.alpha, dy)
    assert torch.equal(dx, dx2) and torch.equal(dalpha, dalpha2)
    keep = live.cpu().numpy()
    X, KK, A, DY = gate_test.f64(x, k, net.alpha, dy)
    (rx, rk, ra), (bx, bk, ba) = gate_test.backward(X[keep], KK[keep], A, DY[keep])
    gx, gk, ga = gate_test.f64(dx, dk, dalpha)
    gate_test.close(gx[keep], rx, bx, True)
    gate_test.close(gk[keep], rk, bk, False)
    gate_test.close(ga, ra, ba, False)
    assert (gx[~keep] == DY[~keep]).all() and not gk[~keep].any()

    # dE = dk wkv: dk in blocks along the hidden columns, wkv^T in the tiles' scales
    wkv_t = np.ascontiguousarray(quantised(net.wkv, 128).T)
    q, s = eg.engram_fp8_quantise(dk)
    w = saved[5]
    de = eg.engram_fp8_matmul(q, s, w[2], w[3], b_block=eg.FP8_BLOCK, out_dtype=torch.bfloat16)
    fp8_test.check_product(de, quantised(dk), wkv_t, True)
    # dwkv = dk^T E: both in blocks along the tokens
    fp8_test.check_product(dwkv, quantised(dk.t()), quantised(e.t()), False)

    uniq, ref, bound = rows_test.reference(ids.cpu().numpy(), de.view(T, -1, net.d).cpu(), net.rows, 1.0, False)
    n = int(count)
    assert n == len(uniq) and (row_ids[:n].cpu().numpy() == uniq).all() and (row_ids[n:] == -1).all()
    rows_test.close(grads[:n].double().cpu().numpy(), ref, bound, "f32")

    gate = 1 / (1 + np.exp(-(X[:, 0] * KK).sum(1) / np.sqrt(((X[:, 0] ** 2).mean(1) + 1e-6)
                                                            * ((KK ** 2).mean(1) + 1e-6) * net.hidden)))
    want = X + (gate * keep)[:, None, None] * KK[:, None] * A[:, None]
    got = y.double().cpu().numpy()
    # the gate off by 2^-12 at most (48 roundings of 2^-24 on a sum of up to 16 in magnitude), then bf16
    tol = 2.0 ** -12 * np.abs(want - X) + 2.0 ** -8 * 1.001 * np.abs(want) + 2.0 ** -133
    assert (np.abs(got - want) <= tol).all()
