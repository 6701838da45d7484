"""fp32 gradients of engram_matmul_grad from an fp32 dy or through an activation: what the products
read of dz keeps 16 bits, not 8.

dz goes in as two bf16 values: the first is at most 2^-8 of dz off, the second at most 2^-8 of what
is left: 2^-16 |dz|.  Otherwise as in tests/test_gpu_matmul.py: (2 length / 16 + 16) 2^-22 of
S = sum |dz b| for the sums (twice the length), 1.2 2^-18 of sum |dy b| for the slope's evaluation,
half a step of the output, a db that is added to another step of the old value.  A bf16 output
beside it keeps its one rounding of dz, 2^-8 S."""
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


def gradients(eg, M, N, K, act, dy="f32", pre="f32", da="f32", db="f32", accumulate=False, layout="rows", pad=0):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + 5 * K)

    def matrix(rows, cols, dtype, turned=False):
        r, c = (cols, rows) if turned else (rows, cols)
        v = torch.full((r, c + pad), float("nan"), device="cuda", dtype=dtype)[:, :c]
        v.copy_(torch.randn(r, c, generator=g, device="cuda"))
        return v.t() if turned else v
    a, b = matrix(M, K, torch.bfloat16, layout != "rows"), matrix(N, K, torch.bfloat16, layout != "rows")
    y = matrix(M, N, dt[dy])
    z = matrix(M, N, dt[pre]) if act != "none" else None
    old = matrix(N, K, dt[db]) if accumulate else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return eg.engram_matmul_grad(y, a, b, pre=z, activation=ACTS.index(act), scale=0.5, accumulate=accumulate,
                                     da_dtype=dt[da], db_dtype=dt[db], db=old.clone() if accumulate else None,
                                     status=status)[:2]
    got = call()
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert all(torch.equal(x, w) for x, w in zip(call(), got))
    dz = y.double() * (slope64(z.double(), act) if z is not None else 1)
    for grad, other, turned, length, kind in ((got[0], b.double(), False, N, da), (got[1], a.double(), True, M, db)):
        d, e = (dz.t(), y.double().t()) if turned else (dz, y.double())
        want, S = 0.5 * (d @ other), 0.5 * (d.abs() @ other.abs())
        slack = ((2 * length / 16 + 16) * 2.0 ** -22 + (2.0 ** -16 if kind == "f32" else 2.0 ** -8)) * S
        if act != "none":
            slack = slack + 1.2 * 2.0 ** -18 * 0.5 * (e.abs() @ other.abs())
        if turned and accumulate:
            want, slack = want + old.double(), slack + 2.0 ** -22 * old.double().abs()
        off = (grad.double() - want).abs() - slack - HALF_STEP[kind] * want.abs()
        assert off.max() <= 0, (kind, float(off.max()))


# A few rows, K shared by CTAs, single tiles, pairs, two products in one launch, odd sizes.
SIZES = [(1, 1, 1), (1, 64, 200), (3, 300, 8), (37, 300, 1300), (300, 257, 260), (130, 2048, 520), (700, 1100, 900),
         (2050, 515, 771), (64, 4096, 1536)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_from_fp32(eg, M, N, K):
    gradients(eg, M, N, K, "none")
    gradients(eg, M, N, K, "none", da="bf16", accumulate=True)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_through_an_activation(eg, M, N, K, act):
    gradients(eg, M, N, K, act)
    gradients(eg, M, N, K, act, dy="bf16", pre="bf16", db="bf16")
    gradients(eg, M, N, K, act, dy="bf16", da="bf16", accumulate=True)


@pytest.mark.parametrize("layout", ["rows", "columns"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_layouts(eg, layout, pad):
    for M, N, K in ((2, 130, 96), (40, 264, 1500), (300, 264, 520), (1500, 1100, 264)):
        gradients(eg, M, N, K, "silu", layout=layout, pad=pad)


def test_long_sums(eg):
    gradients(eg, 20000, 130, 264, "gelu", accumulate=True)


def test_parts_agree(eg):
    """da or db alone, and an exact bf16 dy, whose second values are zeros.  A product alone may share
    K among CTAs where two in a launch do not, and then adds the same values in another order: each is
    within the sums' (2 length / 16 + 16) 2^-22 S of the other's exact value and rounds once more."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    a, b, y = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((300, 136), (200, 136), (300, 200)))
    f32 = dict(da_dtype=torch.float32, db_dtype=torch.float32)
    noise = y.float() + 2.0 ** -12 * torch.randn(300, 200, generator=g, device="cuda")
    da, db, _ = eg.engram_matmul_grad(noise, a, b, **f32)
    d = noise.double().abs() * (1 + 2.0 ** -7)  # the sizes of both values of dz together
    for got, want, S, length in (
            (eg.engram_matmul_grad(noise, a, b, grad_b=False, **f32)[0], da, d @ b.double().abs(), 200),
            (eg.engram_matmul_grad(noise, a, b, grad_a=False, **f32)[1], db, d.t() @ a.double().abs(), 300)):
        slack = 2 * (2 * length / 16 + 16) * 2.0 ** -22 * S + 2.0 ** -23 * want.double().abs()
        assert ((got.double() - want.double()).abs() <= slack).all()
    exact, wide = eg.engram_matmul_grad(y, a, b, **f32), eg.engram_matmul_grad(y.float(), a, b, **f32)
    for got, want, S, length in ((wide[0], exact[0], y.double().abs() @ b.double().abs(), 200),
                                 (wide[1], exact[1], y.double().abs().t() @ a.double().abs(), 300)):
        slack = 2 * (2 * length / 16 + 16) * 2.0 ** -22 * S + 2.0 ** -23 * want.double().abs()
        assert ((got.double() - want.double()).abs() <= slack).all()


def test_values_that_are_not_finite(eg):
    """They reach their own row of da and column of db, with nothing of theirs in the second matrix."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    a, b = (torch.rand(*s, generator=g, device="cuda").bfloat16() + 0.5 for s in ((70, 40), (60, 40)))
    y = torch.rand(70, 60, generator=g, device="cuda") + 0.5
    y[3, 5], y[9, 7] = float("inf"), float("nan")
    da, db, _ = eg.engram_matmul_grad(y, a, b, da_dtype=torch.float32, db_dtype=torch.float32)
    rows, cols = torch.arange(70, device="cuda"), torch.arange(60, device="cuda")
    assert (da[3] == float("inf")).all() and da[9].isnan().all() and da[(rows != 3) & (rows != 9)].isfinite().all()
    assert (db[5] == float("inf")).all() and db[7].isnan().all() and db[(cols != 5) & (cols != 7)].isfinite().all()
