"""engram_matmul and engram_matmul_grad against plain fp64 products.

Tolerance of a product before its epilogue: every a * b is exact in fp32; the tensor cores add
sums of 16 products into an fp32 accumulator, each step off by at most 2^-22 of S = sum |a b|
(a truncation of a value under S, with two bits to spare), and the epilogue's steps by as much:
(K/16 + 16) 2^-22 |scale| S =: t.  Through the activation, whose slope is under 1.13, 1.13 t and
2^-18 (|z| + 2^-4) for its evaluation; each output adds half a step of its type.  The mean over
an output has to look like rounding too: rms error / rms S <= sqrt(K/16 + 16) 2^-22 where nothing
else rounds.  Of the gradient: dz is rounded to bf16 as an operand, half a step 2^-8 of each
|dz|: 2^-8 sum |dz b| on top (and 2^-18 of dy for the slope)."""
import math

import pytest

pytestmark = pytest.mark.gpu
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
ACTS = ["none", "relu", "silu", "gelu"]


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(g, rows, cols, layout="rows", dtype=None, pad=0, offset=0):
    """[rows, cols] values as rows of memory or as columns of it (a transposed view), `pad`
    values between them, starting `offset` values into their buffer."""
    import torch
    r, c = (rows, cols) if layout == "rows" else (cols, rows)
    n = r * (c + pad)
    flat = torch.empty(n + offset, device="cuda", dtype=dtype or torch.bfloat16).fill_(float("nan"))
    v = flat[offset:].view(r, c + pad)[:, :c]
    v.copy_(torch.randn(r, c, generator=g, device="cuda"))
    return v if layout == "rows" else v.t()


def act64(z, act):
    import torch
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z


def slope64(z, act):
    import torch
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def close(got, want, slack, out):
    err = (got.double() - want).abs()
    bad = err > slack + HALF_STEP[out] * want.abs()
    assert not bad.any(), (int(bad.sum()), float((err - slack).max()))


def product(eg, a, b, out="f32", act="none", bias=None, residual=None, scale=1.0, pre=None, dst=None):
    """One call, checked."""
    import torch
    M, K = a.shape
    N = b.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = scale * (a.double() @ b.double().t())
    S = abs(scale) * (a.double().abs() @ b.double().abs().t())
    t = (K / 16 + 16) * 2.0 ** -22 * S
    if bias is not None:
        z = z + bias.double()
        t = t + 2.0 ** -23 * (z.abs() + bias.double().abs())
    keep = None if pre is None else torch.full((M, N), float("nan"), dtype=dt(pre), device="cuda")
    want = act64(z, act)
    slack = t if act == "none" else 1.13 * t + 2.0 ** -18 * (z.abs() + 2.0 ** -4)
    if residual is not None:
        want = want + residual.double()
        slack = slack + 2.0 ** -23 * (want.abs() + residual.double().abs())
    got = eg.engram_matmul(a, b, bias=bias, activation=ACTS.index(act), residual=residual, scale=scale, pre=keep,
                           out=dst, out_dtype=dt(out), status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert got.dtype == dt(out) and got.shape == (M, N)
    close(got, want, slack, out)
    if keep is not None:
        close(keep, z, t, pre)
    if out == "f32" and act == "none" and bias is None and residual is None and M * N * K > 1e6:
        rms = float((got.double() - want).square().mean().sqrt() / S.square().mean().sqrt())
        assert rms <= math.sqrt(K / 16 + 16) * 2.0 ** -22, rms
    return got


# One CTA to a tile, K shared by 2 to 8 CTAs, pairs; odd sizes; lengths of one; several segments.
SIZES = [(1, 1, 1), (1, 16, 8), (3, 1, 70), (1, 4096, 512), (16, 130, 2048), (37, 4096, 640), (128, 128, 64),
         (129, 131, 129), (300, 257, 1000), (1000, 500, 72), (513, 1030, 520), (2050, 700, 1100), (700, 2100, 300),
         (1, 300, 20000), (40, 140, 70000), (1300, 1100, 8300)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_sizes(eg, M, N, K, out):
    g = gen(M + N + K)
    product(eg, matrix(g, M, K), matrix(g, N, K), out)


# K shared by 2 to 8 CTAs: as many of a tile as run at once.
@pytest.mark.parametrize("M,N,K", [(24, 4097, 2100), (37, 4864, 3500), (33, 5500, 2900), (64, 7296, 6144), (20, 9300, 4500),
                                   (60, 5000, 5000), (128, 128, 700), (65, 260, 1290)])
def test_matmul_few_rows_of_many_columns(eg, M, N, K):
    g = gen(M + N + K)
    for out in ("f32", "bf16"):
        product(eg, matrix(g, M, K), matrix(g, N, K), out, act="silu", residual=matrix(g, M, N))


@pytest.mark.parametrize("N,stride", [(5, 8), (9, 16), (33, 64), (191, 192), (185, 192), (252, 256), (1001, 1024)])
@pytest.mark.parametrize("M,K", [(3, 40), (30, 600), (200, 64), (640, 1700)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_leaves_what_lies_beside(eg, M, N, K, stride, out):
    """Rows on 16 bytes that end inside 16 bytes: the values behind them stay, of out, pre and the
    gradients."""
    import torch
    g = gen(M + N)
    mine = {name: torch.full((rows + 1, width), 7.0, dtype=dt(out), device="cuda")
            for name, rows, width in (("out", M, stride), ("pre", M, stride), ("da", M, stride), ("db", K, stride))}
    a, b, r = matrix(g, M, K), matrix(g, N, K), matrix(g, M, N)
    dst = mine["out"][:M, :N]
    product(eg, a, b, out, dst=dst)
    product(eg, a, b, out, act="silu", residual=r, dst=dst)
    dst.copy_(r)
    eg.engram_matmul(a, b, residual=dst, pre=mine["pre"][:M, :N], out=dst)
    close(mine["pre"][:M, :N], a.double() @ b.double().t(), (K / 16 + 16) * 2.0 ** -22 * (a.double().abs() @ b.double().abs().t()), out)
    dy, c = matrix(g, M, K), matrix(g, K, N)
    eg.engram_matmul_grad(dy, r, c, da=mine["da"][:M, :N], db=mine["db"][:K, :N])
    for name, rows in (("out", M), ("pre", M), ("da", M), ("db", K)):
        buf = mine[name].clone()
        assert not (buf[:rows, :N] == 7.0).all()
        buf[:rows, :N] = 7.0
        assert (buf == 7.0).all(), name


@pytest.mark.parametrize("N", [33000, 33001])
def test_offsets_past_32_bits(eg, N):
    """Outputs and gradients of more than 2^31 elements, on 16-byte boundaries and off them."""
    import torch
    M, K = 66000, 40
    g = gen(N)
    a, b = matrix(g, M, K), matrix(g, N, K)
    y = eg.engram_matmul(a, b, out_dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, M // 2, 65074, 65080, M - 2, M - 1], device="cuda")
    want = a[rows].double() @ b.double().t()
    close(y[rows], want, (K / 16 + 16) * 2.0 ** -22 * (a[rows].double().abs() @ b.double().abs().t()), "bf16")
    da, db, dbias = eg.engram_matmul_grad(y, a, b, grad_bias=True, da_dtype=torch.float32, db_dtype=torch.float32)
    z = y[rows].double()
    close(da[rows], z @ b.double(), (N / 16 + 16) * 2.0 ** -22 * (z.abs() @ b.double().abs()), "f32")
    cols = slice(N - 300, N)
    z = y[:, cols].double()
    t = (M / 16 + 16) * 2.0 ** -22
    close(db[cols], z.t() @ a.double(), t * (z.abs().t() @ a.double().abs()), "f32")
    close(dbias[cols], z.sum(0), (M + 4) * 2.0 ** -24 * z.abs().sum(0), "f32")


@pytest.mark.parametrize("M,N,K", [(1, 40, 24), (130, 140, 150), (70, 4100, 1030), (523, 1031, 777), (1024, 1536, 512)])
@pytest.mark.parametrize("a", ["rows", "columns"])
@pytest.mark.parametrize("b", ["rows", "columns"])
def test_matmul_layouts(eg, M, N, K, a, b):
    """Both operands along K or along their rows, padded, off 16-byte boundaries."""
    g = gen(M)
    for pad, offset in ((0, 0), (8, 8), (5, 0), (8, 1)):
        product(eg, matrix(g, M, K, a, pad=pad, offset=offset), matrix(g, N, K, b, pad=pad, offset=offset))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(5, 300, 1100), (200, 333, 90), (600, 1500, 264)])
def test_matmul_epilogues(eg, M, N, K, act):
    """Every type of bias, residual, pre-activation and output."""
    g = gen(N)
    a, b = matrix(g, M, K), matrix(g, N, K)
    one = 1 / math.sqrt(K)
    for out in ("f32", "bf16"):
        for bias in (None, "bf16", "f32"):
            for residual in (None, "bf16", "f32"):
                product(eg, a, b, out, act, bias and matrix(g, 1, N, dtype=dt(bias))[0],
                        residual and matrix(g, M, N, dtype=dt(residual), pad=3), scale=one,
                        pre={None: None, "bf16": "f32", "f32": "bf16"}[residual])


def test_matmul_strided_outputs(eg):
    """Outputs, pre-activation and residual with gaps between their rows, which stay as they are;
    a residual of one row."""
    import torch
    g = gen(3)
    for M, N, K in ((7, 130, 1030), (300, 200, 64), (1000, 600, 128)):
        for out in ("f32", "bf16"):
            a, b = matrix(g, M, K), matrix(g, N, K)
            wide = torch.full((M + 1, N + 5), 7.0, dtype=dt(out), device="cuda")
            row = matrix(g, 1, N, dtype=torch.float32).expand(M, N)
            product(eg, a, b, out, "silu", residual=row, scale=0.1, dst=wide[:M, 2:N + 2])
            assert (wide[M] == 7).all() and (wide[:, :2] == 7).all() and (wide[:, N + 2:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(3, 200, 900), (300, 257, 260), (700, 1100, 17000), (1100, 300, 9000)])
def test_matmul_residual_in_place(eg, M, N, K):
    import torch
    g = gen(K)
    a, b = matrix(g, M, K), matrix(g, N, K)
    for out in ("f32", "bf16"):
        for act in ("none", "gelu"):
            for pre in (None, "f32"):
                x = torch.randn(M, N, generator=g, device="cuda").to(dt(out))
                apart = eg.engram_matmul(a, b, residual=x, activation=ACTS.index(act), scale=0.01, out_dtype=dt(out))
                keep = x.clone()
                z = None if pre is None else torch.empty(M, N, device="cuda")
                eg.engram_matmul(a, b, residual=x, activation=ACTS.index(act), scale=0.01, out=x, pre=z)
                bound = (K / 16 + 16) * 2.0 ** -22 * 0.01 * (a.double().abs() @ b.double().abs().t())
                slack = 2 * HALF_STEP[out] * (apart.double().abs() + keep.double().abs()) + 2.3 * bound
                assert ((x.double() - apart.double()).abs() <= slack).all()


def test_matmul_special_values(eg):
    """Infinities and NaN reach their own outputs, and only those; zeros past the edges of the
    operands do not meet them."""
    import torch
    g = gen(9)
    for M, N, K in ((5, 140, 1000), (140, 150, 70), (600, 1000, 130)):
        a, b = matrix(g, M, K, pad=6), matrix(g, N, K, pad=6)  # the gaps hold NaN
        a[2, 1] = float("nan")
        b[3, 2] = float("inf")
        for act in ("none", "relu"):
            got = eg.engram_matmul(a, b, activation=ACTS.index(act))
            want = a.float() @ b.float().t()
            want = want if act == "none" else torch.relu(want)
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())


def test_matmul_same_bits_and_captured(eg):
    """The same call gives the same bits, alone, among others and from a captured graph."""
    import torch
    g = gen(11)
    for M, N, K in ((16, 300, 2048), (300, 257, 500), (900, 1500, 9000)):
        a, b, x = matrix(g, M, K), matrix(g, N, K), matrix(g, M, N)
        want = eg.engram_matmul(a, b, activation=eg.ACT_SILU, residual=x)
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eg.engram_matmul(a, b, activation=eg.ACT_SILU, residual=x, out=out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
            assert torch.equal(eg.engram_matmul(a, b, activation=eg.ACT_SILU, residual=x), want)


# ----------------------------------------------------------------------------- gradient

def gradient(eg, M, N, K, act="none", dy="bf16", pre="bf16", da="bf16", db="bf16", accumulate=False, scale=1.0,
             layout=("rows", "rows"), pad=0, bias=True):
    import torch
    g = gen(M + 2 * N + 3 * K)
    a, b = matrix(g, M, K, layout[0], pad=pad), matrix(g, N, K, layout[1], pad=pad)
    y = matrix(g, M, N, dtype=dt(dy), pad=pad)
    z = matrix(g, M, N, dtype=dt(pre), pad=pad) if act != "none" else None
    old_b, old_bias = torch.randn(N, K, generator=g, device="cuda").to(dt(db)), torch.randn(N, generator=g, device="cuda")
    got_b, got_bias = (old_b.clone(), old_bias.clone()) if accumulate else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ga, gb, gbias = eg.engram_matmul_grad(y, a, b, pre=z, activation=ACTS.index(act), scale=scale, grad_bias=bias,
                                          accumulate=accumulate, db=got_b, dbias=got_bias if bias else None,
                                          da_dtype=dt(da), db_dtype=dt(db), status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    dz = y.double() * (slope64(z.double(), act) if z is not None else 1)
    rounding = 0.0 if act == "none" and dy == "bf16" else 2.0 ** -8
    slope = 0.0 if act == "none" else 2.0 ** -18 * 1.2
    for got, want, S, length, kind in (
            (ga, dz @ b.double(), dz.abs() @ b.double().abs(), N, da),
            (gb, dz.t() @ a.double(), dz.abs().t() @ a.double().abs(), M, db)):
        want, S = scale * want, abs(scale) * S
        slack = ((length / 16 + 16) * 2.0 ** -22 + rounding) * S
        if slope:
            slack = slack + slope * abs(scale) * (y.double().abs() @ b.double().abs() if got is ga
                                                  else y.double().abs().t() @ a.double().abs())
        if got is gb and accumulate:
            want = want + old_b.double()
            slack = slack + 2.0 ** -22 * old_b.double().abs()
        close(got, want, slack, kind)
    if bias:
        want = dz.sum(0) + (old_bias.double() if accumulate else 0)
        # blocks of rows, each a warp's share of 8 in turn
        slack = (M / 8 + 80) * 2.0 ** -24 * dz.abs().sum(0) + slope * y.double().abs().sum(0) + 2.0 ** -23 * old_bias.abs()
        close(gbias, want, slack, "f32")
    else:
        assert gbias is None


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 1, 1), (37, 300, 130), (300, 1100, 520), (2050, 515, 771)])
def test_gradient(eg, M, N, K, act):
    gradient(eg, M, N, K, act)
    gradient(eg, M, N, K, act, dy="f32", pre="f32", da="f32", db="f32")
    gradient(eg, M, N, K, act, accumulate=True, db="f32", scale=0.5)


@pytest.mark.parametrize("a", ["rows", "columns"])
@pytest.mark.parametrize("b", ["rows", "columns"])
def test_gradient_layouts(eg, a, b):
    for pad in (0, 8, 3):
        gradient(eg, 300, 264, 520, "gelu", layout=(a, b), pad=pad)
        gradient(eg, 301, 265, 523, "none", layout=(a, b), pad=pad, db="f32", bias=False)


def test_gradient_long_sums(eg):
    """A weight gradient over many tokens, and added to the last one's, in fp32."""
    gradient(eg, 40000, 130, 264, db="f32")
    gradient(eg, 20000, 700, 520, db="f32", accumulate=True)


def test_gradient_parts(eg):
    """Only what is asked for; rows of dy that repeat; no tokens at all."""
    import torch
    g = gen(21)
    a, b, y = matrix(g, 300, 130), matrix(g, 200, 130), matrix(g, 300, 200)
    both = eg.engram_matmul_grad(y, a, b, grad_bias=True)
    for parts in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        some = eg.engram_matmul_grad(y, a, b, grad_a=parts[0], grad_b=parts[1], grad_bias=parts[2])
        for asked, got, want in zip(parts, some, both):
            assert (got is not None) == asked and (got is None or torch.equal(got, want))
    row = y[:1].expand(300, 200)
    for got, want in zip(eg.engram_matmul_grad(row, a, b, grad_bias=True),
                         eg.engram_matmul_grad(row.contiguous(), a, b, grad_bias=True)):
        assert torch.equal(got, want)
    kept = torch.ones(200, 130, device="cuda")
    da, db, dbias = eg.engram_matmul_grad(y[:0], a[:0], b, grad_bias=True)
    assert da.shape == (0, 130) and not db.any() and not dbias.any()
    eg.engram_matmul_grad(y[:0], a[:0], b, db=kept, accumulate=True)
    assert (kept == 1).all()


def test_gradient_against_differences(eg):
    """sum(dy * out) moves with a weight, an input and a bias as the gradient says: central
    differences of the fp32 outputs.  out is smooth: a step of h leaves h^2 of its third
    derivatives, and the difference 2^-21 sum |dy out| / h of rounding."""
    import torch
    g = gen(31)
    M, N, K = 40, 48, 64
    a, b, y = matrix(g, M, K), matrix(g, N, K), matrix(g, M, N)
    bias, x = torch.randn(N, generator=g, device="cuda"), matrix(g, M, N)
    scale, h = 0.125, 2.0 ** -5
    for act in ("silu", "gelu"):
        z = torch.empty(M, N, device="cuda")

        def loss(a, b, bias):
            out = eg.engram_matmul(a, b, bias=bias, activation=ACTS.index(act), residual=x, scale=scale, pre=z)
            return float((y.double() * out.double()).sum()), float((y.double() * out.double()).abs().sum())
        loss(a, b, bias)
        da, db, dbias = eg.engram_matmul_grad(y, a, b, pre=z, activation=ACTS.index(act), scale=scale, grad_bias=True,
                                              da_dtype=torch.float32, db_dtype=torch.float32)
        for which, grad, at in ((0, da, (3, 5)), (1, db, (7, 9)), (2, dbias, (11,))):
            args = [a.float(), b.float(), bias.clone()]
            v = float(args[which][at])
            step = 2.0 ** -3 if which < 2 else h  # values that bf16 holds
            ends = []
            for sign in (1, -1):
                moved = [t.clone() for t in args]
                moved[which][at] = v + sign * step
                moved = [moved[0].bfloat16(), moved[1].bfloat16(), moved[2]]
                ends.append((loss(*moved), float(moved[which][at])))
            (up, mag), at_up = ends[0]
            (down, _), at_down = ends[1]
            difference = (up - down) / (at_up - at_down)
            width = (at_up - at_down) / 2
            # third derivatives of silu and gelu are under 1.3; the slack for dz's rounding 2^-8
            other = {0: (y.double().abs()[at[0]] * b.double()[:, at[1]].abs() if which == 0 else None),
                     1: (y.double().abs()[:, at[0]] * a.double()[:, at[1]].abs() if which == 1 else None),
                     2: (y.double().abs()[:, at[0]] if which == 2 else None)}[which]
            lever = {0: scale * float(b.float()[:, at[-1]].abs().max()), 1: scale * float(a.float()[:, at[-1]].abs().max()),
                     2: 1.0}[which]
            weight = float(other.sum()) * (scale if which < 2 else 1.0)
            slack = weight * (2.0 ** -8 * 1.2 + 1.3 * (lever * width) ** 2 / 6) + 2.0 ** -21 * mag / width
            assert abs(difference - float(grad[at])) <= slack, (act, which)
