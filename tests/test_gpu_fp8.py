"""engram_fp8_quantise, bit for bit against the definition, and engram_fp8_matmul against a
plain fp64 product.

The quantised bytes and scales are whole numbers with one right answer: the reference finds
the scale with frexp on exact fp64 values and rounds on the list of e4m3 values itself.

Product tolerance: every a * b * 2^(ea + eb) is exact in fp32; the tensor cores add K/32
partial sums of 32 products into an fp32 accumulator, each step off by at most one fp32
rounding of a value bounded by S = sum |a b|.  Allowing 2^-22 per step and 16 steps more:
(K/32 + 16) 2^-22 S, plus 2^-8 of the value where the output is bf16.  On average the
errors must look like rounding, not like a wrong term: their rms over S stays within
sqrt(K/32 + 16) 2^-23 (fp32 outputs)."""
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def e4m3_values():
    """The value of each byte, from the format's definition."""
    b = np.arange(256)
    s, e, m = np.where(b & 128, -1.0, 1.0), b >> 3 & 15, b & 7
    v = s * np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[127] = v[255] = np.nan
    return v


VALUES = e4m3_values()
GRID = VALUES[:127]  # non-negative, ascending, its index the byte


def round_e4m3(v):
    """The nearest byte of |v| <= 448 with v's sign, ties to the even byte."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(GRID, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - GRID[lo], GRID[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def reference(x, br):
    """(bytes, scale bytes) of fp64 x [M, K]."""
    M, K = x.shape
    q = np.empty((M, K), np.uint8)
    s = np.empty((-(-M // br), -(-K // 128)), np.uint8)
    for kb in range(s.shape[1]):
        cols = slice(kb * 128, kb * 128 + 128)
        for mb in range(s.shape[0]):
            rows = slice(mb * br, mb * br + br)
            blk = x[rows, cols]
            if not np.isfinite(blk).all():
                s[mb, kb], q[rows, cols] = 255, 127
                continue
            big = np.abs(blk).max()
            e = -127
            if big > 0:
                m, ex = np.frexp(big / 448.0)        # big = 448 m 2^ex, 1/2 <= m < 1
                e = max(-127, ex - 1 if m == 0.5 else ex)
            s[mb, kb] = e + 127
            q[rows, cols] = round_e4m3(blk * 2.0 ** -e)
    return q, s


def awkward(M, K, dtype, seed):
    """Values over the whole range: blocks of their own size, exact ties, zeros, subnormals."""
    import torch
    r = np.random.default_rng(seed)
    x = r.standard_normal((M, K)) * np.exp2(r.integers(-30, 30, (M, 1)))
    x[r.random((M, K)) < 0.05] = 0
    x[::5] = GRID[r.integers(0, 127, x[::5].shape)] * 2.0 ** -20             # on the grid
    mid = (GRID[:-1] + GRID[1:]) / 2
    x[1::5] = -mid[r.integers(0, 126, x[1::5].shape)] * 2.0 ** 11            # ties
    x[2::17] = 0.0
    x[3::17] *= 2.0 ** -140                                                  # fp32 subnormals
    x[4::17] *= 2.0 ** 90
    x[6::17, ::3] = -0.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


QCASES = [(1, 1), (1, 128), (3, 16), (5, 200), (37, 6144), (128, 128), (129, 257), (300, 1000),
          (16, 4096), (260, 384), (1000, 127), (4099, 24)]


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", QCASES)
def test_quantise_is_the_definition(eg, M, K, dtype, br):
    import torch
    x = awkward(M, K, {"bf16": torch.bfloat16, "f32": torch.float32}[dtype], seed=M + K)
    v = x.double().numpy()
    rq, rs = reference(v, br)
    rqt, rst = reference(np.ascontiguousarray(v.T), br)
    for rows, cols in ((True, False), (False, True), (True, True)):
        out = eg.engram_fp8_quantise(x.cuda(), block_rows=br, rows=rows, cols=cols)
        want = ([rq, rs] if rows else []) + ([rqt, rst] if cols else [])
        assert len(out) == len(want)
        for got, ref in zip(out, want):
            assert np.array_equal(got.cpu().numpy(), ref)


def test_quantise_scale_boundaries(eg):
    """Maxima at and next to 448 * 2^e, for every exponent of fp32, alone in their block."""
    import torch
    edges = np.array([448 * 2.0 ** e for e in range(-126, 119)], np.float32)
    pts = np.concatenate([edges, np.nextafter(edges, np.float32(0)), np.nextafter(edges, np.float32(np.inf)),
                          np.array([np.finfo(np.float32).max, 1e-45, 2.0 ** -126, 0], np.float32)])
    x = np.zeros((len(pts), 128), np.float32)
    x[np.arange(len(pts)), np.arange(len(pts)) % 128] = -pts
    q, s = eg.engram_fp8_quantise(torch.from_numpy(x).cuda())
    rq, rs = reference(x.astype(np.float64), 1)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("br", [1, 128])
def test_quantise_non_finite_blocks(eg, br):
    import torch
    x = torch.ones(140, 300)
    x[3, 5], x[4, 140], x[5, 299], x[139, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    for rows, cols in ((True, False), (True, True)):
        out = eg.engram_fp8_quantise(x.cuda(), block_rows=br, rows=rows, cols=cols)
        v = x.double().numpy()
        want = reference(v, br) + (reference(np.ascontiguousarray(v.T), br) if cols else ())
        for got, ref in zip(out, want):
            assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("cols", [False, True])
def test_quantise_strides_leave_the_padding(eg, cols):
    """x a slice of wider rows (odd stride and start), q and qt slices with padding kept."""
    import torch
    M, K = 70, 150
    base = awkward(M, K + 7, torch.float32, 5).cuda()
    x = base[:, 3:3 + K]
    buf, tbuf = torch.full((M, 192), 7, dtype=torch.uint8, device="cuda"), torch.full((K, 96), 7, dtype=torch.uint8, device="cuda")
    s, st = (torch.empty(n, 2 if n == M else 1, dtype=torch.uint8, device="cuda") for n in (M, K))
    eg.engram_fp8_quantise(x, cols=cols, out=[buf[:, :K], s] + ([tbuf[:, :M], st] if cols else []))
    v = x.double().cpu().numpy()
    rq, rs = reference(v, 1)
    assert np.array_equal(buf[:, :K].cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    assert (buf[:, K:] == 7).all()
    if cols:
        rqt, rst = reference(np.ascontiguousarray(v.T), 1)
        assert np.array_equal(tbuf[:, :M].cpu().numpy(), rqt) and np.array_equal(st.cpu().numpy(), rst)
    assert (tbuf[:, M:] == 7).all()


# ------------------------------------------------------------------------- product

def operand(eg, rows, K, block, seed, lo=110, hi=140):
    """Random bytes (no NaN) and scale bytes; the operand's fp64 values."""
    import torch
    r = np.random.default_rng(seed)
    q = r.integers(0, 256, (rows, K)).astype(np.uint8)
    q[(q & 127) == 127] = 0
    s = r.integers(lo, hi, (-(-rows // block), -(-K // 128))).astype(np.uint8)
    dev = eg.fp8_empty(rows, K, "cuda")
    dev.copy_(torch.from_numpy(q))
    wide = np.exp2(s.astype(np.float64) - 127).repeat(128, 1)[:, :K]
    return dev, torch.from_numpy(s).cuda(), VALUES[q] * wide.repeat(block, 0)[:rows]


def check_product(got, av, bv, bf16):
    import torch
    a, b = torch.from_numpy(av).cuda(), torch.from_numpy(bv).cuda()
    ref, S = a @ b.t(), a.abs() @ b.abs().t()
    K = a.shape[1]
    err = (got.double() - ref).abs()
    tol = (K / 32 + 16) * 2.0 ** -22 * S
    if bf16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -133
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())
    if not bf16:
        rms = float((err / S.clamp(min=1e-300)).square().mean().sqrt())
        assert rms <= (K / 32 + 16) ** 0.5 * 2.0 ** -23


MCASES = [(1, 1, 1), (1, 128, 128), (16, 16, 16), (7, 100, 130), (16, 4096, 6144), (1, 640, 2048),
          (33, 257, 1000), (64, 512, 512), (128, 128, 512), (129, 129, 129), (200, 1000, 640),
          (256, 256, 384), (300, 70, 4096), (1000, 1030, 1100), (2500, 2300, 300), (5, 9000, 256),
          (9000, 5, 256), (512, 4096, 6144), (257, 2048, 8200),
          (1601, 1600, 640), (4100, 1100, 9000), (1900, 2049, 8320), (20000, 260, 1500), (16411, 256, 16)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("blocks", [(1, 128), (1, 1), (128, 128), (128, 1)])
@pytest.mark.parametrize("M,N,K", MCASES)
def test_product_matches_fp64(eg, M, N, K, blocks, out):
    import torch
    a, sa, av = operand(eg, M, K, blocks[0], M + K)
    b, sb, bv = operand(eg, N, K, blocks[1], N + K + 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    got = eg.engram_fp8_matmul(a, sa, b, sb, *blocks, out_dtype=dt, status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    assert got.dtype == dt
    check_product(got, av, bv, out == "bf16")
    again = eg.engram_fp8_matmul(a, sa, b, sb, *blocks, out_dtype=dt)
    assert torch.equal(got, again)


def test_product_of_whole_numbers_is_exact(eg):
    """Small integers with scales that make one block count 1, the next 2, 4, ...: every sum
    is exact, so a scale read from the wrong row, block or byte shows."""
    import torch
    M, N, K = 300, 400, 128 * 11
    r = np.random.default_rng(3)
    av, bv = r.integers(-4, 5, (M, K)), r.integers(-4, 5, (N, K))
    lut = {float(v): i for i, v in reversed(list(enumerate(VALUES))) if v == v}
    enc = np.vectorize(lambda v: lut[float(v)], otypes=[np.uint8])
    sa = r.integers(0, 4, (M, 11)).astype(np.uint8)
    sb = r.integers(0, 4, (N, 11)).astype(np.uint8)
    a, b = eg.fp8_empty(M, K, "cuda"), eg.fp8_empty(N, K, "cuda")
    a.copy_(torch.from_numpy(enc(av)))
    b.copy_(torch.from_numpy(enc(bv)))
    got = eg.engram_fp8_matmul(a, torch.from_numpy(sa + 127).cuda(), b, torch.from_numpy(sb + 127).cuda())
    ref = (av * 2 ** sa.astype(np.int64).repeat(128, 1)) @ (bv * 2 ** sb.astype(np.int64).repeat(128, 1)).T
    assert np.array_equal(got.cpu().numpy(), ref.astype(np.float32))


def test_product_strides(eg):
    """Operands and output that are slices of wider buffers; nothing beside them is read into
    the sums or written."""
    import torch
    M, N, K = 50, 75, 300
    a, sa, av = operand(eg, M, K, 1, 1)
    b, sb, bv = operand(eg, N, K, 1, 2)
    wa = torch.full((M, 336), 0x7F, dtype=torch.uint8, device="cuda")   # NaN beside the rows
    wb = torch.full((N, 400), 0x7F, dtype=torch.uint8, device="cuda")
    wa[:, 16:16 + K], wb[:, :K] = a, b
    buf = torch.full((M, N + 3), 5.0, device="cuda")
    eg.engram_fp8_matmul(wa[:, 16:16 + K], sa, wb[:, :K], sb, out=buf[:, 1:1 + N])
    check_product(buf[:, 1:1 + N], av, bv, False)
    assert (buf[:, 0] == 5.0).all() and (buf[:, 1 + N:] == 5.0).all()


def test_product_nan_stays_in_its_rows(eg):
    import torch
    M, N, K = 40, 300, 512
    a, sa, av = operand(eg, M, K, 1, 1)
    b, sb, bv = operand(eg, N, K, 1, 2)
    a[3, 500], sb[200, 1], a[7, 0] = 0x7F, 0xFF, 0xFF
    got = eg.engram_fp8_matmul(a, sa, b, sb)
    bad_m, bad_n = [3, 7], [200]
    assert got[bad_m].isnan().all() and got[:, bad_n].isnan().all()
    keep_m = [i for i in range(M) if i not in bad_m]
    keep_n = [i for i in range(N) if i not in bad_n]
    check_product(got[keep_m][:, keep_n], av[keep_m], bv[keep_n], False)


def test_product_of_quantised_values(eg):
    """quantise then multiply, both copies of x: x w^T along K and x^T y along the rows."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(333, 700, generator=g, device="cuda")
    w = torch.randn(250, 700, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn(333, 90, generator=g, device="cuda")
    q, s, qt, st = eg.engram_fp8_quantise(x, cols=True)
    qw, sw = eg.engram_fp8_quantise(w, block_rows=128)
    qyt, syt = eg.engram_fp8_quantise(y, rows=False, cols=True)

    def value(q, s, br=1):
        wide = np.exp2(s.cpu().numpy().astype(np.float64) - 127).repeat(128, 1)[:, :q.shape[1]]
        return VALUES[q.cpu().numpy()] * wide.repeat(br, 0)[:q.shape[0]]
    check_product(eg.engram_fp8_matmul(q, s, qw, sw, b_block=128), value(q, s), value(qw, sw, 128), False)
    check_product(eg.engram_fp8_matmul(qt, st, qyt, syt), value(qt, st), value(qyt, syt), False)


def test_product_empty(eg):
    import torch
    a, sa, _ = operand(eg, 5, 64, 1, 1)
    e, se = eg.fp8_empty(0, 64, "cuda"), torch.empty(0, 1, dtype=torch.uint8, device="cuda")
    assert eg.engram_fp8_matmul(e, se, a, sa).shape == (0, 5)
    assert eg.engram_fp8_matmul(a, sa, e, se).shape == (5, 0)
    assert [tuple(t.shape) for t in eg.engram_fp8_quantise(torch.empty(0, 64, device="cuda"), cols=True)] == \
        [(0, 64), (0, 1), (64, 0), (64, 0)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(512, 1024, 8192), (16, 6144, 4096), (371, 260, 12052), (151, 5888, 8320),
                                   (53, 1283, 12462), (2100, 1500, 8320), (405, 128, 5120), (241, 2300, 16400)])
def test_product_long_sums_and_few_tiles(eg, M, N, K, out):
    """K shared by the CTAs of a cluster, and K in several accumulators, at every kind of tile."""
    test_product_matches_fp64(eg, M, N, K, (1, 128), out)
