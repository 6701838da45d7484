"""engram_embed against a plain fp64 lookup: types, pooled and not, widths from one
column, strided ids, tables and outputs, dead and bad ids, empty calls.

Tolerance: bf16 and fp32 values are exact in fp32, so an unpooled value is one product,
rounded once to fp32 (2^-24 of it) and, for bf16, once more (2^-8, half an ulp of its
8-bit significand); a pooled one adds R terms in fp32 first (2^-24 of the sum of their
magnitudes each)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def make(T, R, D, rows, table, seed, dead=0.2):
    import torch
    g = np.random.default_rng(seed)
    t = torch.from_numpy(g.standard_normal((rows, D)).astype(np.float32)).to(_dt(table))
    ids = g.integers(0, rows, (T, R)).astype(np.int32)
    ids[g.random((T, R)) < dead] = -1
    return t, ids


def reference(t, ids, scale, pooled):
    """(value, sum of magnitudes) in fp64."""
    v = np.vstack([t.double().numpy(), np.zeros((1, t.shape[1]))])[ids]  # -1: the zero row
    v = v * float(np.float32(scale))
    return (v.sum(1), np.abs(v).sum(1)) if pooled else (v, np.abs(v))


def check(got, ref, mag, R, out, pooled):
    import torch
    got = got.double().cpu().numpy()
    n = R + 1 if pooled else 1
    tol = n * 2.0 ** -24 * mag + (2.0 ** -8 * mag * n * 2.0 ** -24 + 2.0 ** -8 * np.abs(ref) * 1.001
                                  if out == "bf16" else 0) + 2.0 ** -133
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) - tol)


CASES = [(1, 1, 1), (1, 1, 4096), (3, 2, 7), (5, 1, 16), (37, 6, 256), (129, 24, 8), (1000, 3, 250),
         (64, 9, 1000), (2, 24, 4104), (700, 24, 256), (4000, 1, 264), (3, 1, 16384)]


@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,R,D", CASES)
def test_embed_matches_fp64(eg, T, R, D, table, out, pooled):
    t, ids = make(T, R, D, 97, table, seed=T * 1000 + R * 10 + D)
    import torch
    got = eg.engram_embed(torch.from_numpy(ids).cuda(), t.cuda(), scale=0.37, pooled=pooled,
                          out_dtype=_dt(out))
    ref, mag = reference(t, ids, 0.37, pooled)
    assert got.shape == ref.shape and got.dtype == _dt(out)
    check(got, ref, mag, R, out, pooled)


def test_embed_scale_one_copies_bits(eg):
    import torch
    t = torch.arange(65536, dtype=torch.int32).to(torch.int16).reshape(256, 256)
    ids = torch.arange(255, -1, -1, dtype=torch.int32)
    got = eg.engram_embed(ids.cuda(), t.cuda(), out=torch.empty(256, 256, dtype=torch.int16, device="cuda"))
    want = t[ids.long()]
    nan = (want & 0x7F80) == 0x7F80  # a NaN's payload is not part of its value
    nan &= (want & 0x7F) != 0
    got = got.cpu()
    assert torch.equal(got[~nan], want[~nan])
    assert (((got[nan] & 0x7F80) == 0x7F80) & ((got[nan] & 0x7F) != 0)).all()


@pytest.mark.parametrize("D,pad,off", [(64, 8, 0), (64, 3, 1), (33, 7, 2)])
def test_embed_strides_and_alignment(eg, D, pad, off):
    """Ids that are a slice of wider rows, a table and an output with padded, shifted rows:
    the concatenated rows of one order inside [tokens, 3 H D]."""
    import torch
    T, R = 50, 4
    t, ids = make(T, R, D, 61, "bf16", seed=D + pad)
    wide = torch.full((T, 3 * R), -7, dtype=torch.int32, device="cuda")
    wide[:, R:2 * R] = torch.from_numpy(ids)
    tab = torch.zeros(61 * (D + pad) + off, dtype=torch.bfloat16, device="cuda")
    tv = tab[off:].view(61, D + pad)[:, :D]
    tv.copy_(t)
    buf = torch.full((T, 3 * R * D + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, R * D:2 * R * D].unflatten(1, (R, D))
    got = eg.engram_embed(wide[:, R:2 * R], tv, scale=2.0, out=out)
    ref, mag = reference(t, ids, 2.0, False)
    check(got, ref, mag, R, "bf16", False)
    buf[:, R * D:2 * R * D] = 5.0
    assert (buf == 5.0).all()  # nothing beside the slice was written


@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("D", [8, 31])
def test_embed_bad_ids_flag_and_stay_unwritten(eg, D, pooled):
    import torch
    t, ids = make(20, 3, D, 50, "f32", seed=5, dead=0.0)
    ids[4, 1], ids[7, 0], ids[9, 2] = 50, -2, 2 ** 31 - 1
    ids[11] = -1
    bad = [(4, 1), (7, 0), (9, 2)]
    out = torch.full((20, D) if pooled else (20, 3, D), 123.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_embed(torch.from_numpy(ids).cuda(), t.cuda(), pooled=pooled, out=out, status=status)
    assert eg.engram_read_status(status) == (eg.ERR_OUT_OF_RANGE, eg.FLAG_BAD_ROW)
    safe = ids.copy()
    for r, c in bad:
        safe[r, c] = 0
    ref, mag = reference(t, safe, 1.0, pooled)
    got = out.double().cpu().numpy()
    for r, c in bad:
        at = r if pooled else (r, c)
        assert (got[at] == 123.0).all()
        ref[at] = mag[at] = 123.0
    check(torch.from_numpy(got), ref, mag, 3, "f32", pooled)
    assert (got[11] == 0).all()


def test_embed_empty(eg):
    import torch
    t = torch.zeros(4, 8, device="cuda")
    for shape in ((0,), (0, 3)):
        out = eg.engram_embed(torch.zeros(shape, dtype=torch.int32, device="cuda"), t)
        assert out.shape == (*shape, 8)


def test_embed_offsets_beyond_32_bits(eg):
    """A row whose byte offset needs 33 bits, in a table of 2 GiB + a row of bf16 values."""
    import torch
    rows, D = (1 << 31) // 256 + 3, 256
    t = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    t[-1] = torch.arange(D, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([0, rows - 1, rows - 2], dtype=torch.int32, device="cuda")
    got = eg.engram_embed(ids, t)
    assert torch.equal(got[1], t[-1]) and not got[0].any() and not got[2].any()


def test_embed_runs_on_the_given_stream(eg):
    """The call is ordered on the stream it is given, not on torch's current one."""
    import torch
    t, ids = make(2000, 24, 256, 97, "bf16", seed=1)
    tc, ic = t.cuda(), torch.from_numpy(ids).cuda()
    want = eg.engram_embed(ic, tc)
    s = torch.cuda.Stream()
    late = torch.zeros_like(tc)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(tc, non_blocking=True)
    eg.engram_embed(ic, late, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,R,D,pad", [(9801, 24, 256, 0), (6601, 24, 64, 8), (79001, 2, 32, 0), (2503, 24, 1024, 16)])
def test_embed_many_rows(eg, T, R, D, pad, table, out):
    """Lists long enough for the form that takes 32 rows a warp, compared on the device."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    rows, scale = 1001, 0.37
    t = torch.randn(rows, D + pad, device="cuda", generator=g).to(_dt(table))[:, :D]
    ids = torch.randint(-1, rows, (T, R), device="cuda", generator=g, dtype=torch.int32)
    ids[T - 1] = -1
    ids[:, 1] = torch.where(ids[:, 1] % 7 == 3, rows + ids[:, 1], ids[:, 1])  # bad ones
    got = torch.full((T, R, D + pad), 9.0, dtype=_dt(out), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_embed(ids, t, scale=scale, out=got[..., :D], status=status)
    assert eg.engram_read_status(status)[1] == eg.FLAG_BAD_ROW
    assert (got[..., D:] == 9.0).all()
    for a in range(0, T, 2000):  # in slices: fp64
        i, y = ids[a:a + 2000].long(), got[a:a + 2000, :, :D].double()
        ref = t.double()[i.clamp(0, rows - 1)] * float(np.float32(scale)) * (i >= 0).unsqueeze(-1)
        tol = 2.0 ** -24 * ref.abs() + 2.0 ** -133
        if out == "bf16":
            tol = tol + 2.0 ** -8 * 1.001 * ref.abs()
        bad = (i >= rows).unsqueeze(-1).expand_as(y)
        assert (torch.where(bad, y == 9.0, (y - ref).abs() <= tol)).all()


@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,R,D,pad", [(5003, 1, 17, 0), (2600, 2, 33, 1), (811, 6, 109, 0), (5001, 1, 66, 3),
                                       (1700, 3, 250, 0), (2503, 2, 475, 2), (204, 24, 1278, 0), (4865, 1, 256, 1)])
def test_embed_many_unaligned_rows(eg, T, R, D, pad, table, out):
    if R == 1:  # the check below writes bad ids into the second column
        T, R = T // 2 + 1, 2
    test_embed_many_rows(eg, T, R, D, pad, table, out)
