"""The training example as a whole: its gradients against torch's in fp32 on the same chain
without quantisation, loosely, and its loss, which has to fall.  Each link on its own operands
is in test_gpu_train_connection_operands.py."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location(
        "train_connection", os.path.join(ROOT, "examples", "train_connection.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_follow_the_unquantised_chain(example):
    """An e4m3 value is within 2^-4 of what it stands for (3 stored bits, to nearest) while that is
    at least 2^-13 of the block's largest magnitude, and within 2^-17 of that magnitude below
    (e4m3's subnormals), so each product of two such factors is about within 2^-3 + 2^-8 of
    the plain one, term by term, and over many terms of either sign the errors average out: the
    norm of a gradient's error stays well inside 2^-3 of its own norm, and its direction within a
    cosine of 0.99."""
    import torch
    net = example.Connection(seed=3)
    T = 700
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, net.n_eids, (1, T), generator=g, device="cuda", dtype=torch.int32)
    dead = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    dead[0, ::9] = 1
    x = torch.randn(T, 4, net.hidden, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, 4, net.hidden, generator=g, device="cuda").bfloat16()
    ids = net.row_ids(tokens, dead)
    y, saved = net.forward(ids, x)
    dx, dalpha, dwkv, (row_ids, grads, count) = net.backward(saved, dy)

    table = net.table.float().requires_grad_()
    wkv, alpha = net.wkv.clone().requires_grad_(), net.alpha.clone().requires_grad_()
    xs = x.float().requires_grad_()
    live = (ids[:, :1] >= 0).float()
    e = (table[ids.long().clamp(min=0)] * (ids >= 0).unsqueeze(-1)).view(T, net.K)
    k = e @ wkv.t()
    D = net.hidden
    ra = (xs[:, 0].square().mean(1, keepdim=True) + 1e-6).rsqrt()
    rk = (k.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    gate = torch.sigmoid((xs[:, 0] * k).sum(1, keepdim=True) * ra * rk / D ** 0.5) * live
    out = xs + (gate * k).unsqueeze(1) * alpha.view(1, 4, 1)
    out.backward(dy.float())
    out = out.detach()

    def near(got, ref, name):
        got, ref = got.double(), ref.double()
        assert float((got - ref).norm() / ref.norm()) < 0.125, name
        assert float((got * ref).sum() / (got.norm() * ref.norm())) > 0.99, name
    near(y.float() - x.float(), out - x.float(), "the memory's contribution")
    near(dx.float() - dy.float(), xs.grad - dy.float(), "dx")
    near(dalpha, alpha.grad, "dalpha")
    near(dwkv, wkv.grad, "dwkv")
    n = int(count)
    dense = torch.zeros_like(table)
    dense[row_ids[:n].long()] = grads[:n]
    near(dense, table.grad, "dtable")
    assert not (row_ids[:n] < 0).any() and (row_ids[n:] == -1).all()


def test_loss_falls(example):
    losses = example.train(tokens=2048, steps=20)
    assert losses[-1] < 0.9 * losses[0] and all(b < a for a, b in zip(losses, losses[1:6]))
