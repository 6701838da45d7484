"""Activations and their slopes far from zero, in fp32, against fp64: right to their own size, not
only to that of 1.

K = 1, b = 1 and bf16 values z make pre exactly z.  Tolerances in steps of 2^-24 of the value.  The
normal distribution below z < 0 is e^(-z^2/2) G(-z): __expf is off by 2 + 1.173 z^2/2 units in the last
place (2 steps each), its argument's rounding moves it by z^2/2 steps, G is off by 4.4e-7 (8 steps), and
six steps for the products.  silu(z) = z / (1 + e^-z): __expf 2 + 1.173 |z| units, the sum and the
quotient 4 units more.  The slopes are compared to the sum of their terms' sizes: of gelu Phi(z) and
z phi(z), each as above; of silu s (1 + z (1 - s)) four more operations on s, which is right as the
quotient above.  z stays over -12: below, gelu leaves fp32's normal numbers soon."""
import math

import pytest

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def values():
    import torch
    return torch.cat([torch.linspace(-12, 12, 389), torch.tensor([-5.0, -1e-3, 0.0, 1e-3, 40.0, 300.0])]).cuda().bfloat16()


# By warps, clusters or single CTAs and pairs; the last with rows off 16 bytes.
@pytest.mark.parametrize("M,N", [(4, 395), (40, 395), (395, 40), (395, 512), (395, 41), (5135, 2048)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations(eg, act, M, N):
    import torch
    z = values()
    along = M % 395 == 0  # the values go along a's rows or along b's
    a, b = (z.repeat(M // 395)[:, None], torch.ones(N, 1)) if along else (torch.ones(M, 1), z[:, None])
    out = eg.engram_matmul(a.bfloat16().cuda(), b.bfloat16().cuda(),
                           activation=getattr(eg, "ACT_" + act.upper())).double()
    d = (a.double().cuda() @ b.double().cuda().t())
    if act == "gelu":
        want = d / 2 * torch.special.erfc(-d / math.sqrt(2))
        slack = 4 + (1.173 + 0.5) * d * d + 8 + 6
    else:
        want = d * torch.sigmoid(d)
        slack = 2 * (2 + 1.173 * d.abs()) + 8
    assert ((out - want).abs() <= slack * STEP * want.abs()).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes(eg, act):
    import torch
    z = values()
    one = torch.ones(395, 1, dtype=torch.bfloat16, device="cuda")
    a = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    pre = z[None].float()
    _, _, dbias = eg.engram_matmul_grad(torch.ones(1, 395, device="cuda"), a, one, pre=pre, grad_bias=True,
                                        activation=getattr(eg, "ACT_" + act.upper()))
    d = z.double()
    if act == "gelu":
        phi = d * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
        below = torch.special.erfc(-d / math.sqrt(2)) / 2
        want = below + phi
        slack = (4 + (1.173 + 0.5) * d * d + 8 + 6) * (below + phi.abs())
    else:
        s = torch.sigmoid(d)
        want = s * (1 + d * (1 - s))
        slack = (2 * (2 + 1.173 * d.abs()) + 16) * s * (1 + d.abs())
    assert ((dbias.double() - want).abs() <= slack * STEP).all()
