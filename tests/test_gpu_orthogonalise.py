"""engram_orthogonalise against the iteration in fp64.

The kernels round the iterate and the two square matrices to fp16 (11 bits) between products;
sums are fp32.  `rounded` is the same iteration in fp64 with those roundings, E its distance from
the iteration without any.  The kernels' roundings fall in the same places on sums that differ
by fp32 rounding, so their error is another draw of the same size: 2 E is allowed, and half a
step of bf16, 2^-8 of each value, for the result.  Sides under 16 have few roundings to average:
there the worst case is allowed.  With the usual coefficients a relative error e of A, B and X
each step moves a singular value s <= 1.3 by at most e (|b| s^3 + 2 c s^5 + |B| s + s) <= 26 e;
e = 2^-11, five steps, each damped by the next (the slope of the iteration at the values it
settles among, 0.7 to 1.2, is under 1.3 in magnitude on average): 26 * 5 * 2^-11."""
import math

import pytest

pytestmark = pytest.mark.gpu
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def iterate(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, half=False):
    """The iteration in fp64 on [M, N]; `half` with the roundings to fp16."""
    import torch

    def r(t):
        return (t * 256).half().double() / 256 if half else t
    a, b, c = coefficients
    x = r(u.double() / (u.double().square().sum().sqrt() + eps))
    tall = x.shape[0] > x.shape[1]
    for i in range(steps):
        gram = r(x.t() @ x if tall else x @ x.t())
        q = r(b * gram + c * (gram @ gram))
        x = a * x + (x @ q if tall else q @ x)
        x = x if i == steps - 1 else r(x)
    return x


def check(got, u, scale=1.0, **kw):
    import torch
    want = iterate(u, **kw)
    E = float((iterate(u, half=True, **kw) - want).norm())
    norm = float(want.norm())
    slack = 2 * E + 2.0 ** -8 * norm
    if min(u.shape) < 16:
        slack = max(slack, 26 * 5 * 2.0 ** -11 * norm)
    off = float((got.double() / scale - want).norm())
    assert got.dtype == torch.bfloat16 and off <= slack, (off / norm, E / norm)


def gradients(g, L, M, N, dtype):
    import torch
    x = torch.randn(L, M, N, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(L, M, 1, generator=g, device="cuda"))
    low = torch.randn(L, M, 3, generator=g, device="cuda") @ torch.randn(L, 3, N, generator=g, device="cuda")
    return (1e-3 * (x + low)).to(dtype)


# Wide, tall and square; odd sides; sides of one; every form of the products.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 37), (37, 1), (2, 3), (16, 16), (17, 130), (130, 17), (64, 257),
                                 (128, 64), (128, 3584), (3584, 128), (100, 3585), (90, 700), (1000, 129), (128, 449),
                                 (256, 1536), (475, 300), (300, 475), (513, 1030), (1030, 513), (1100, 1100),
                                 (2100, 700), (700, 2100)])
def test_sizes(eg, M, N, dtype):
    import torch
    g = gradients(gen(M + N), 1, M, N, {"bf16": torch.bfloat16, "f32": torch.float32}[dtype])[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = eg.engram_orthogonalise(g, status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0) and out.shape == (M, N)
    check(out, g)


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("L,M,N", [(1, 65, 200), (3, 200, 65), (12, 130, 260), (40, 16, 24), (200, 40, 300), (40, 20, 1800)])
def test_momentum_and_batches(eg, L, M, N, nesterov):
    """Several steps of several matrices at once: the momentum is beta m + g in fp32, one rounding
    of the sum (fma); every matrix has its own update."""
    import torch
    g = gen(L)
    m = 3e-3 * torch.randn(L, M, N, generator=g, device="cuda")
    for step in range(3):
        x = gradients(g, L, M, N, torch.float32)
        want = (0.9 * m.double() + x.double())
        out = eg.engram_orthogonalise(x, momentum=m, beta=0.9, nesterov=nesterov, scale=0.2)
        # 0.9 as fp32 is 2^-26 off; half a step of the result
        assert ((m.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -25 * want.abs().max()).all()
        u = x.double() + 0.9 * m.double() if nesterov else m.double()
        for i in range(L):
            check(out[i], u[i], scale=0.2)


def test_values(eg):
    """Singular values come near one, directions stay."""
    import torch
    g = gen(5)
    for M, N in ((300, 1000), (1000, 300)):
        x = torch.randn(M, N, generator=g, device="cuda")
        out = eg.engram_orthogonalise(x).double()
        s = torch.linalg.svdvals(out)
        assert 0.6 < s.min() and s.max() < 1.3
        U, _, V = torch.linalg.svd(x.double(), full_matrices=False)
        inner = (U.t() @ out @ V.t())
        assert (inner - torch.diag(inner.diagonal())).abs().max() < 0.02 and inner.diagonal().min() > 0.6


def test_options(eg):
    """Other coefficients and numbers of steps: the cubic iteration converges to one."""
    import torch
    x = torch.randn(130, 300, generator=gen(6), device="cuda")
    for steps in (1, 2, 12, 20):
        check(eg.engram_orthogonalise(x, steps=steps, coefficients=(1.5, -0.5, 0.0), eps=0.0), x, steps=steps,
              coefficients=(1.5, -0.5, 0.0), eps=0.0)
    s = torch.linalg.svdvals(eg.engram_orthogonalise(x, steps=20, coefficients=(1.5, -0.5, 0.0)).double())
    assert (s - 1).abs().max() < 0.02


def test_strides(eg):
    """Gaps between rows and matrices, which stay as they are; any alignment."""
    import torch
    for L, M, N in ((2, 70, 130), (3, 131, 50)):
        for dtype in (torch.bfloat16, torch.float32):
            g = gen(N)
            wide = torch.full((L, M + 2, N + 3), float("nan"), dtype=dtype, device="cuda")
            x = wide[:, 1:M + 1, 1:N + 1]
            x.copy_(gradients(g, L, M, N, dtype))
            mom = torch.full((L, M + 1, N + 1), 5.0, device="cuda")
            m = mom[:, :M, :N]
            m.copy_(1e-3 * torch.randn(L, M, N, generator=g, device="cuda"))
            dst = torch.full((L, M + 1, N + 5), 7.0, dtype=torch.bfloat16, device="cuda")
            m2 = m.clone()
            want = eg.engram_orthogonalise(x.contiguous(), momentum=m2)
            got = eg.engram_orthogonalise(x, momentum=m, out=dst[:, :M, 3:N + 3])
            assert torch.equal(got, want) and torch.equal(m, m2)
            assert (mom[:, M] == 5).all() and (mom[:, :, N] == 5).all()
            assert (dst[:, M] == 7).all() and (dst[:, :, :3] == 7).all() and (dst[:, :, N + 3:] == 7).all()
            one = eg.engram_orthogonalise(x[1], momentum=torch.zeros(M, N, device="cuda"))
            check(one, x[1].double() * 1.95)


@pytest.mark.parametrize("L,M,N,stride", [(2, 60, 91, 96), (2, 129, 191, 192), (1, 333, 210, 216), (3, 130, 1001, 1024)])
def test_leaves_what_lies_beside(eg, L, M, N, stride):
    import torch
    x = gradients(gen(3), L, M, N, torch.float32)
    out = torch.full((L, M + 1, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    eg.engram_orthogonalise(x, out=out[:, :M, :N])
    assert torch.equal(out[:, :M, :N], eg.engram_orthogonalise(x))
    out[:, :M, :N] = 7.0
    assert (out == 7.0).all()


def test_special_matrices(eg):
    """Zeros stay zero, one entry alone stays one, a NaN is its own matrix's; tiny and huge
    gradients come out as others do."""
    import torch
    x = torch.randn(5, 90, 70, generator=gen(7), device="cuda")
    plain = eg.engram_orthogonalise(x, eps=0.0)
    y = x.clone()
    y[1] = 0
    y[2, 3, 4] = float("nan")
    y[3, 0, 0] = float("inf")
    y[4] *= 2.0 ** 40
    out = eg.engram_orthogonalise(y)
    assert not out[1].any() and out[2].isnan().all() and out[3].isnan().any()
    assert torch.equal(out[4], plain[4]) and torch.equal(eg.engram_orthogonalise(x * 2.0 ** -40, eps=0.0), plain)
    alone = torch.zeros(64, 100, device="cuda")
    alone[5, 6] = -3.0
    got = eg.engram_orthogonalise(alone).double()
    want = iterate(torch.full((1, 1), 3.0, device="cuda"))[0, 0]
    assert abs(float(got[5, 6] + want)) < 0.03 and (got != 0).sum() == 1


def test_no_matrices(eg):
    import torch
    assert eg.engram_orthogonalise(torch.zeros(0, 4, 5, device="cuda")).shape == (0, 4, 5)


def test_same_bits_and_captured(eg):
    """The same bits from every call and from a captured graph, beside another graph."""
    import torch
    for L, M, N in ((1, 300, 500), (7, 130, 70)):
        x = gradients(gen(8), L, M, N, torch.float32)
        want = eg.engram_orthogonalise(x)
        outs = [torch.empty_like(want) for _ in range(2)]
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        for graph, out in zip(graphs, outs):
            with torch.cuda.graph(graph):
                eg.engram_orthogonalise(x, out=out)
        for _ in range(3):
            for graph, out in zip(graphs, outs):
                out.zero_()
                graph.replay()
            assert all(torch.equal(out, want) for out in outs) and torch.equal(eg.engram_orthogonalise(x), want)


def test_training_run(eg):
    """A two-layer block trained for three steps -- product with bias and activation, product
    with residual, gradients, updates -- link by link against fp64 on each link's own operands."""
    import torch
    g = gen(9)
    T, D, H = 300, 256, 520
    w1, w2 = ((torch.randn(*s, generator=g, device="cuda") / 16).bfloat16() for s in ((H, D), (D, H)))
    b1, b2 = torch.zeros(H, device="cuda"), torch.zeros(D, device="cuda")
    m1, m2 = torch.zeros(H, D, device="cuda"), torch.zeros(D, H, device="cuda")

    def near(got, want, S, length, bits=2.0 ** -8):
        assert ((got.double() - want).abs() <= bits * want.abs() + ((length / 16 + 16) * 2.0 ** -22 + 2.0 ** -8) * S).all()
    for step in range(3):
        x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
        target = torch.randn(T, D, generator=g, device="cuda")
        z = torch.empty(T, H, device="cuda")
        h = eg.engram_matmul(x, w1, bias=b1, activation=eg.ACT_GELU, pre=z, out_dtype=torch.bfloat16)
        y = eg.engram_matmul(h, w2, bias=b2, residual=x)
        near(z, x.double() @ w1.double().t() + b1, x.double().abs() @ w1.double().t().abs(), D)
        near(h, torch.nn.functional.gelu(z.double()), z.double().abs(), 0)
        near(y, h.double() @ w2.double().t() + b2 + x.double(), h.double().abs() @ w2.double().t().abs(), H)
        dy = (y - target) / T
        dh, dw2, db2 = eg.engram_matmul_grad(dy, h, w2, grad_bias=True, db_dtype=torch.float32)
        dx, dw1, db1 = eg.engram_matmul_grad(dh, x, w1, pre=z, activation=eg.ACT_GELU, grad_bias=True,
                                             db_dtype=torch.float32)
        zd = z.double().requires_grad_()
        (slope,) = torch.autograd.grad(torch.nn.functional.gelu(zd).sum(), zd)
        dz = dh.double() * slope
        near(dw2, dy.double().t() @ h.double(), dy.double().t().abs() @ h.double().abs(), T)
        near(dh, dy.double() @ w2.double(), dy.double().abs() @ w2.double().abs(), D)
        near(dw1, dz.t() @ x.double(), dz.t().abs() @ x.double().abs(), T)
        near(dx, dz @ w1.double(), dz.abs() @ w1.double().abs(), H)
        near(db1, dz.sum(0), dz.abs().sum(0), T)
        near(db2, dy.double().sum(0), dy.double().abs().sum(0), T)
        for w, m, b, dw, db in ((w1, m1, b1, dw1, db1), (w2, m2, b2, dw2, db2)):
            update = eg.engram_orthogonalise(dw, momentum=m, scale=0.2 * math.sqrt(max(w.shape)))
            check(update, dw.double() + 0.95 * m.double(), scale=0.2 * math.sqrt(max(w.shape)))
            w.sub_(update, alpha=0.01)
            b.sub_(db, alpha=0.01)
