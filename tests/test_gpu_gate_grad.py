"""engram_gate_add_grad against the formula in fp64 and against differences of the
forward pass in fp64: widths, dead and bad tokens, in place, both dk types.

Tolerances, written out in bounds(): a dot of D products is a tree of at most 48 fp32
additions deep (8 a thread, 5 shuffles, 32 warps); that error, e(x, y) = 48 * 2^-24 *
sum |x y|, is carried through z, the gate and its slope to first order and doubled;
elementwise sums add 8 roundings of their terms' magnitudes; bf16 outputs round once
more (2^-8, half an ulp of its 8-bit significand)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
EPS = 1e-6
U = 2.0 ** -24


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def forward(x, k, alpha):
    """out [T, 4, D] in fp64 (not rounded)."""
    D = k.shape[1]
    a = x[:, 0]
    ra = 1 / np.sqrt((a * a).mean(1) + EPS)
    rk = 1 / np.sqrt((k * k).mean(1) + EPS)
    g = 1 / (1 + np.exp(-ra * rk * (a * k).sum(1) / np.sqrt(D)))
    return x + (g[:, None] * k)[:, None, :] * alpha[:, None]


def backward(x, k, alpha, dy):
    """The formula in fp64, and per output the bound on an fp32 evaluation's error."""
    D = k.shape[1]
    a = x[:, 0]
    dot = lambda p, q: (p * q).sum(1)  # noqa: E731
    e = lambda p, q: 48 * U * (np.abs(p) * np.abs(q)).sum(1)  # noqa: E731
    ra, rk = 1 / np.sqrt(dot(a, a) / D + EPS), 1 / np.sqrt(dot(k, k) / D + EPS)
    u = ra * rk / np.sqrt(D)
    z = dot(a, k) * u
    g = 1 / (1 + np.exp(-z))
    slope = g * (1 / (1 + np.exp(z)))
    dyk = (dy * k[:, None, :]).sum(2)
    e_dyk = 48 * U * (np.abs(dy) * np.abs(k[:, None, :])).sum(2)
    dc = dyk @ alpha
    dz = dc * slope
    c = np.einsum("tsd,s->td", dy, alpha)
    col = lambda v: v[:, None]  # noqa: E731
    dk = col(g) * c + col(dz * u) * a - col(dz * z * rk * rk / D) * k
    dx = dy.copy()
    dx[:, 0] += col(dz * u) * k - col(dz * z * ra * ra / D) * a
    dalpha = (g[:, None] * dyk).sum(0)
    # bounds
    rel = 64 * U                                    # of ra, rk and of u
    ez = u * e(a, k) + np.abs(z) * 2 * rel
    eg_ = 0.25 * ez + 4 * U * g
    es = 0.1 * ez + 8 * U * slope
    edc = e_dyk @ np.abs(alpha) + 6 * U * np.abs(dyk) @ np.abs(alpha)
    edz = np.abs(dc) * es + slope * edc + 2 * U * np.abs(dz)
    cabs = np.einsum("tsd,s->td", np.abs(dy), np.abs(alpha))

    def side(p, q, w):  # error and magnitude of dz (u p - z w q / D)
        err = col(edz) * (col(u) * np.abs(p) + col(np.abs(z) * w / D) * np.abs(q)) \
            + col(np.abs(dz) * ez * w / D) * np.abs(q)
        mag = col(np.abs(dz) * u) * np.abs(p) + col(np.abs(dz * z) * w / D) * np.abs(q)
        return err + 4 * rel * mag, mag
    err_k, mag_k = side(a, k, rk * rk)
    err_x, mag_x = side(k, a, ra * ra)
    bk = 2 * (err_k + col(eg_) * cabs + 8 * U * (mag_k + col(g) * cabs))
    bx = np.zeros_like(dx)
    bx[:, 0] = 2 * (err_x + 8 * U * (mag_x + np.abs(dy[:, 0])))
    T = len(z)
    ba = 2 * ((np.abs(dyk) * eg_[:, None] + g[:, None] * e_dyk).sum(0)
              + (T + 16) * U * np.abs(g[:, None] * dyk).sum(0))
    return (dx, dk, dalpha), (bx, bk, ba)


def make(T, D, seed):
    import torch
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((T, 4, D)).astype(np.float32)).to(torch.bfloat16)
    mix = (3 / np.sqrt(D) * r.standard_normal((T, 1))).astype(np.float32)
    k = torch.from_numpy(r.standard_normal((T, D)).astype(np.float32) + mix * x[:, 0].float().numpy())
    dy = torch.from_numpy((r.standard_normal((T, 4, D)) * np.exp(r.standard_normal((T, 1, 1))))
                          .astype(np.float32)).to(torch.bfloat16)
    alpha = torch.from_numpy(r.standard_normal(4).astype(np.float32))
    return x, k, dy, alpha


def f64(*ts):
    return [t.double().cpu().numpy() for t in ts]


def close(got, ref, bound, bf16):
    tol = bound + (2.0 ** -8 * (np.abs(ref) + bound) * 1.001 + 2.0 ** -133 if bf16 else 2.0 ** -140)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (bad.mean(), np.max(np.abs(got - ref) / (tol + 1e-300)))


CASES = [(1, 16), (3, 48), (300, 16), (257, 128), (100, 256), (65, 272), (40, 1000 // 16 * 16), (1, 4096),
         (700, 4096), (5, 4112), (33, 8192), (5000, 64)]


@pytest.mark.parametrize("dk_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", CASES)
def test_matches_the_formula(eg, T, D, dk_dtype):
    import torch
    x, k, dy, alpha = make(T, D, seed=T + D)
    dt = torch.bfloat16 if dk_dtype == "bf16" else torch.float32
    dx, dk, da = eg.engram_gate_add_grad(k.cuda(), None, x.cuda(), alpha.cuda(), dy.cuda(), eps=EPS,
                                         dk_dtype=dt)
    (rx, rk, ra), (bx, bk, ba) = backward(*f64(x, k, alpha), dy.double().numpy())
    gx, gk, ga = f64(dx, dk, da)
    close(gx, rx, bx, True)
    close(gk, rk, bk, dk_dtype == "bf16")
    close(ga, ra, ba, False)
    assert (gx[:, 1:] == rx[:, 1:]).all()


@pytest.mark.parametrize("D", [32, 512])
def test_dead_bad_and_in_place(eg, D):
    import torch
    T = 130
    x, k, dy, alpha = make(T, D, seed=9)
    state = torch.zeros(T, dtype=torch.uint8)
    state[::7], state[3::11] = 1, 2
    k[3::11] = float("nan")  # what a bad token holds is not read into anything
    x[3::11] = float("inf")
    live = (state == 0).numpy()
    fill = torch.full_like(dy, 9.0).cuda()
    dx, dk, da = eg.engram_gate_add_grad(k.cuda(), state.cuda(), x.cuda(), alpha.cuda(), dy.cuda(),
                                         eps=EPS, dx=fill)
    (rx, rk, ra), (bx, bk, ba) = backward(*(v[live] for v in f64(x, k)), *f64(alpha), f64(dy)[0][live])
    gx, gk, ga = f64(dx, dk, da)
    close(gx[live], rx, bx, True)
    close(gk[live], rk, bk, False)
    close(ga, ra, ba, False)
    st = state.numpy()
    assert (gk[~live] == 0).all()
    assert (gx[st == 1] == f64(dy)[0][st == 1]).all()
    assert (gx[st == 2] == 9.0).all()
    again = dy.cuda()
    dx2, dk2, da2 = eg.engram_gate_add_grad(k.cuda(), state.cuda(), x.cuda(), alpha.cuda(), again,
                                            eps=EPS, dx=again)
    assert torch.equal(dk2, dk) and torch.equal(da2, da)  # the same bits
    keep = torch.from_numpy(st != 2).cuda()
    assert torch.equal(dx2[keep], dx[keep]) and torch.equal(dx2[~keep].cpu(), dy[st == 2])


def test_all_tokens_dead_and_no_tokens(eg):
    import torch
    x, k, dy, alpha = make(10, 64, seed=2)
    dead = torch.ones(10, dtype=torch.uint8, device="cuda")
    dx, dk, da = eg.engram_gate_add_grad(k.cuda(), dead, x.cuda(), alpha.cuda(), dy.cuda())
    assert torch.equal(dx.cpu(), dy) and not dk.any() and not da.any()
    da = torch.full((4,), 7.0, device="cuda")
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    eg.engram_gate_add_grad(torch.empty(0, 64, device="cuda"), None, e, alpha.cuda(), e.clone(), dalpha=da)
    assert not da.any()


def test_saturated_gates_and_zero_memory(eg):
    """z of +-64 (k = +-stream 0): the slope underflows smoothly; k = 0 has no direction."""
    import torch
    D = 4096
    x, k, dy, alpha = make(3, D, seed=3)
    k[0], k[1], k[2] = x[0, 0].float(), -x[1, 0].float(), 0
    dx, dk, da = eg.engram_gate_add_grad(k.cuda(), None, x.cuda(), alpha.cuda(), dy.cuda(), eps=EPS)
    (rx, rk, ra), (bx, bk, ba) = backward(*f64(x, k, alpha), dy.double().numpy())
    gx, gk, ga = f64(dx, dk, da)
    close(gx, rx, bx, True)
    close(gk, rk, bk, False)
    close(ga, ra, ba, False)


def test_matches_differences(eg):
    """<gradient, v> against (L(p + h v) - L(p - h v)) / 2h of the fp64 forward pass, L =
    <out, dy>: the gradient's own fp32 error, the difference's h^2 term and its rounding
    (1e-16 L / h) are all far below 1e-5 of |gradient| |v|."""
    import torch
    T, D, h = 6, 128, 1e-4
    x, k, dy, alpha = make(T, D, seed=4)
    # stream gradients that bf16 holds as the formula gives them would round: use dk and
    # dalpha in fp32, and dx - dy's direction through stream 0 with dy's own rounding added
    dx, dk, da = eg.engram_gate_add_grad(k.cuda(), None, x.cuda(), alpha.cuda(), dy.cuda(), eps=EPS)
    X, K, A, DY = f64(x, k, alpha, dy)
    GX, GK, GA = f64(dx, dk, da)
    r = np.random.default_rng(8)
    loss = lambda X, K, A: (forward(X, K, A) * DY).sum()  # noqa: E731
    for which, G, slack in (("k", GK, 1e-5), ("a", GA, 1e-5), ("x", GX, 2.0 ** -8)):
        P = {"k": K, "a": A, "x": X}[which]
        for _ in range(4):
            v = r.standard_normal(P.shape)
            up, down = {"k": K, "a": A, "x": X}, {"k": K, "a": A, "x": X}
            up[which], down[which] = P + h * v, P - h * v
            diff = (loss(up["x"], up["k"], up["a"]) - loss(down["x"], down["k"], down["a"])) / (2 * h)
            assert abs((G * v).sum() - diff) <= slack * np.linalg.norm(G) * np.linalg.norm(v)


@pytest.mark.parametrize("dk_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(700, 4112), (500, 8192), (1300, 512), (900, 6000)])
def test_several_tokens_a_block(eg, T, D, dk_dtype):
    test_matches_the_formula(eg, T, D, dk_dtype)


@pytest.mark.parametrize("D", [4096, 4112, 8192])
def test_dead_bad_and_in_place_wide(eg, D):
    test_dead_bad_and_in_place(eg, D)


def test_wide_dead_tokens_among_many(eg):
    import torch
    T, D = 1000, 4224
    x, k, dy, alpha = make(T, D, seed=4)
    state = (torch.arange(T) % 3 == 1).to(torch.uint8)
    live = state == 0
    dx, dk, da = eg.engram_gate_add_grad(k.cuda(), state.cuda(), x.cuda(), alpha.cuda(), dy.cuda(), eps=EPS)
    ox, ok, oa = eg.engram_gate_add_grad(k[live].cuda(), None, x[live].cuda(), alpha.cuda(), dy[live].cuda(),
                                         eps=EPS)
    assert torch.equal(dx.cpu()[live], ox.cpu()) and torch.equal(dk.cpu()[live], ok.cpu())
    assert torch.equal(dx.cpu()[~live], dy[~live]) and not dk.cpu()[~live].any()
    assert torch.allclose(da, oa, rtol=1e-4, atol=1e-3 * float(da.abs().max()))
