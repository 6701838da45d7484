"""engram_embed_grad and engram_embed_grad_rows against a plain fp64 scatter-add: lists from
one id to many tiles of the sort, all ids equal to all different, dead and bad ids, pooled
and not, dense, accumulated and sparse.

Tolerance: a row that c ids name is a sum of c fp32 terms (exact inputs) in some order, so
it is within (c + 4) 2^-24 of the sum of its terms' magnitudes; scaled, rounded once more,
and for bf16 once more still (2^-8)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


def make_ids(T, R, rows, kind, seed):
    r = np.random.default_rng(seed)
    if kind == "uniform":
        ids = r.integers(0, rows, (T, R))
    elif kind == "equal":
        ids = np.full((T, R), rows - 1)
    elif kind == "distinct":
        ids = r.permutation(max(rows, T * R))[:T * R].reshape(T, R) % rows
    else:  # a few rows take most of it, some tokens dead
        ids = np.minimum((rows * r.random((T, R)) ** 6).astype(np.int64), rows - 1)
        ids[r.random(T) < 0.2] = -1
    return ids.astype(np.int32)


def make_dy(T, R, D, dtype, pooled, seed):
    import torch
    r = np.random.default_rng(seed + 1)
    shape = (T, D) if pooled else (T, R, D)
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(_dt(dtype))


def reference(ids, dy, rows, scale, pooled):
    """(gradient, bound without the output's rounding) over the rows that appear, ascending."""
    T, R = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    d = dy.double().numpy()
    if pooled:
        d = np.repeat(d, R, axis=0)
    d = d.reshape(T * R, -1)
    keep = (flat >= 0) & (flat < rows)
    uniq, inv, cnt = np.unique(flat[keep], return_inverse=True, return_counts=True)
    order = np.argsort(inv, kind="stable")
    d = d[keep][order]
    at = np.r_[0, np.cumsum(cnt)[:-1]] if len(cnt) else np.zeros(0, np.int64)
    scale = float(np.float32(scale))
    if len(cnt) == 0:
        return uniq, np.zeros((0, d.shape[1])), np.zeros((0, d.shape[1]))
    g = np.add.reduceat(d, at, axis=0) * scale
    m = np.add.reduceat(np.abs(d), at, axis=0) * abs(scale)
    return uniq, g, (cnt[:, None] + 4) * U * m


def close(got, ref, bound, out):
    tol = bound + 2.0 ** -140
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -133
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (bad.mean(), np.abs(got - ref)[bad].max())


CASES = [  # T, R, D, rows, kind
    (1, 1, 1, 1, "equal"), (1, 1, 4096, 5, "uniform"), (3, 2, 8, 1, "equal"), (37, 6, 33, 50, "uniform"),
    (256, 6, 256, 4096, "uniform"), (130, 24, 64, 3000, "distinct"), (4096, 1, 16, 4096, "distinct"),
    (4097, 1, 24, 300, "skewed"), (1500, 3, 1000, 700, "skewed"), (700, 24, 256, 100003, "skewed"),
    (20000, 1, 40, 3, "uniform"), (9000, 2, 7, 70000, "skewed"), (5000, 1, 4096, 129280 // 8, "skewed"),
    (30000, 3, 8, 1, "equal"), (6000, 1, 520, 2, "equal"), (50, 9, 16384, 40, "uniform"),
]


@pytest.mark.parametrize("dy_dtype,out", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("T,R,D,rows,kind", CASES)
def test_matches_fp64(eg, T, R, D, rows, kind, pooled, dy_dtype, out):
    import torch
    ids = make_ids(T, R, rows, kind, seed=T + D)
    dy = make_dy(T, R, D, dy_dtype, pooled, seed=T + D)
    uniq, ref, bound = reference(ids, dy, rows, 0.37, pooled)
    ci, cd = torch.from_numpy(ids).cuda(), dy.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grad = torch.full((rows, D), float("nan"), dtype=_dt(out), device="cuda")
    eg.engram_embed_grad(ci, cd, rows, scale=0.37, pooled=pooled, grad=grad, status=status)
    full, fb = np.zeros((rows, D)), np.zeros((rows, D))
    full[uniq], fb[uniq] = ref, bound
    close(grad.double().cpu().numpy(), full, fb, out)
    grads = torch.full((T * R, D), 7.0, dtype=_dt(out), device="cuda")
    row_ids, grads, count = eg.engram_embed_grad_rows(ci, cd, rows, scale=0.37, pooled=pooled, grads=grads,
                                                      status=status)
    assert eg.engram_read_status(status) == (eg.OK, 0)
    n = int(count)
    got_ids = row_ids.cpu().numpy()
    assert n == len(uniq) and (got_ids[:n] == uniq).all() and (got_ids[n:] == -1).all()
    close(grads[:n].double().cpu().numpy(), ref, bound, out)
    assert (grads[n:] == 7.0).all()
    assert torch.equal(grads[:n], grad[torch.from_numpy(uniq).cuda()])  # both forms: the same bits


@pytest.mark.parametrize("kind", ["skewed", "equal"])
def test_is_deterministic(eg, kind):
    import torch
    ids = torch.from_numpy(make_ids(3000, 8, 5000, kind, 3)).cuda()
    dy = make_dy(3000, 8, 128, "f32", False, 3).cuda()
    first = eg.engram_embed_grad(ids, dy, 5000)
    for _ in range(5):
        assert torch.equal(eg.engram_embed_grad(ids, dy, 5000), first)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T", [60, 5000])
def test_accumulate_adds_and_leaves_other_rows(eg, T, out):
    import torch
    rows, D = 900, 48
    ids, dy = make_ids(T, 2, rows, "skewed", T), make_dy(T, 2, D, "bf16", False, T)
    old = torch.randn(rows, D, generator=torch.Generator().manual_seed(1)).to(_dt(out))
    old[0, 0] = -0.0
    uniq, ref, bound = reference(ids, dy, rows, 1.0, False)
    grad = old.cuda()
    eg.engram_embed_grad(torch.from_numpy(ids).cuda(), dy.cuda(), rows, grad=grad, accumulate=True)
    want, fb = old.double().numpy().copy(), np.zeros((rows, D))
    want[uniq] += ref
    fb[uniq] = bound + 2 * U * (np.abs(want[uniq]) + np.abs(ref) + bound)
    close(grad.double().cpu().numpy(), want, fb, out)
    other = np.setdiff1d(np.arange(rows), uniq)
    bits = torch.int32 if out == "f32" else torch.int16
    assert torch.equal(grad.cpu().view(bits)[other], old.view(bits)[other])


@pytest.mark.parametrize("T", [40, 6000])
def test_bad_ids_flag_and_take_no_part(eg, T):
    import torch
    rows, D = 64, 16
    ids, dy = make_ids(T, 1, rows, "uniform", 1), make_dy(T, 1, D, "f32", False, 1)
    ids[3], ids[5], ids[T - 1], ids[8] = rows, -2, 2 ** 31 - 1, -2 ** 31
    uniq, ref, bound = reference(ids, dy, rows, 1.0, False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    row_ids, grads, count = eg.engram_embed_grad_rows(torch.from_numpy(ids).cuda(), dy.cuda(), rows, status=status)
    assert eg.engram_read_status(status) == (eg.ERR_OUT_OF_RANGE, eg.FLAG_BAD_ROW)
    n = int(count)
    assert (row_ids[:n].cpu().numpy() == uniq).all()
    close(grads[:n].double().cpu().numpy(), ref, bound, "f32")


@pytest.mark.parametrize("T", [50, 5000])
def test_all_dead_and_empty(eg, T):
    import torch
    ids = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    dy = torch.full((T, 2, 8), float("nan"), device="cuda")  # a dead id's gradient is not read into anything
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert not eg.engram_embed_grad(ids, dy, 33, status=status).any()
    row_ids, _, count = eg.engram_embed_grad_rows(ids, dy, 33, status=status)
    assert int(count) == 0 and (row_ids == -1).all()
    assert eg.engram_read_status(status) == (eg.OK, 0)
    e = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    grad = torch.ones(33, 8, device="cuda")
    eg.engram_embed_grad(e, torch.empty(0, 2, 8, device="cuda"), 33, grad=grad)
    assert not grad.any()
    count = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    eg.engram_embed_grad_rows(e, torch.empty(0, 2, 8, device="cuda"), 33, count=count)
    assert int(count) == 0


@pytest.mark.parametrize("D,pad,off", [(64, 8, 0), (64, 3, 1), (30, 2, 2)])
def test_strides_broadcast_and_alignment(eg, D, pad, off):
    """One order's ids out of a [tokens, 3R] array; dy a slice of a wider, shifted buffer, then a
    row broadcast over a token's ids; a gradient with padded rows."""
    import torch
    T, R, rows = 300, 4, 90
    ids = make_ids(T, R, rows, "uniform", 7)
    wide = torch.full((T, 3 * R), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, R:2 * R] = torch.from_numpy(ids)
    dy = make_dy(T, R, D, "bf16", False, 7)
    buf = torch.full((T * (3 * R * D + pad) + off,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = buf[off:].view(T, 3 * R * D + pad)[:, R * D:2 * R * D].unflatten(1, (R, D))
    view.copy_(dy)
    gbuf = torch.full((rows * (D + pad) + off,), 5.0, device="cuda")
    grad = gbuf[off:].view(rows, D + pad)[:, :D]
    eg.engram_embed_grad(wide[:, R:2 * R], view, rows, scale=2.0, grad=grad)
    uniq, ref, bound = reference(ids, dy, rows, 2.0, False)
    full, fb = np.zeros((rows, D)), np.zeros((rows, D))
    full[uniq], fb[uniq] = ref, bound
    close(grad.double().cpu().numpy(), full, fb, "f32")
    assert (gbuf[off:].view(rows, D + pad)[:, D:] == 5.0).all()
    one = make_dy(T, R, D, "f32", True, 8)
    a = eg.engram_embed_grad(wide[:, R:2 * R], one.cuda().unsqueeze(1).expand(T, R, D), rows)
    b = eg.engram_embed_grad(wide[:, R:2 * R], one.cuda(), rows, pooled=True)
    assert torch.equal(a, b)


def test_largest_ids_sparse(eg):
    """Ids up to 2^31 - 2: four passes of the sort, keys of 31 bits."""
    import torch
    rows = 2 ** 31 - 1
    r = np.random.default_rng(0)
    for T in (100, 9000):
        ids = r.integers(0, rows, (T, 1)).astype(np.int32)
        ids[: T // 2] = rows - 1 - ids[: T // 2] % 50
        dy = make_dy(T, 1, 16, "f32", False, T)
        uniq, ref, bound = reference(ids, dy, rows, 1.0, False)
        row_ids, grads, count = eg.engram_embed_grad_rows(torch.from_numpy(ids).cuda(), dy.cuda(), rows)
        n = int(count)
        assert (row_ids[:n].cpu().numpy() == uniq).all()
        close(grads[:n].double().cpu().numpy(), ref, bound, "f32")


def test_dense_offsets_beyond_32_bits(eg):
    import torch
    rows, D = (1 << 31) // 256 + 5, 256
    ids = torch.tensor([rows - 1, 3, rows - 1, rows - 4], dtype=torch.int32, device="cuda")
    dy = torch.ones(4, D, device="cuda")
    grad = torch.full((rows, D), 1.0, dtype=torch.bfloat16, device="cuda")
    eg.engram_embed_grad(ids, dy, rows, grad=grad)
    assert (grad[-1] == 2).all() and (grad[3] == 1).all() and (grad[-4] == 1).all()
    grad[-1], grad[3], grad[-4] = 0, 0, 0
    assert not grad.any()


@pytest.mark.parametrize("pooled", [False, True])
def test_is_the_lookups_adjoint(eg, pooled):
    """The lookup is linear in its table, so its difference in a direction v is the lookup of v:
    <grad, v> = <embed(v), dy>, in fp64 from the two calls' fp32 outputs.  A sum of c terms is
    off by c 2^-24 of their magnitudes, and no row here is named by more than 32 ids: 2^-19 a
    side."""
    import torch
    T, R, D, rows = 400, 6, 72, 500
    ids = torch.from_numpy(make_ids(T, R, rows, "uniform", 2)).cuda()
    dy = make_dy(T, R, D, "f32", pooled, 2).cuda()
    v = torch.randn(rows, D, generator=torch.Generator().manual_seed(3)).cuda()
    grad = eg.engram_embed_grad(ids, dy, rows, scale=0.5, pooled=pooled)
    y = eg.engram_embed(ids, v, scale=0.5, pooled=pooled)
    mag = float((eg.engram_embed(ids, v.abs(), scale=0.5, pooled=pooled).double() * dy.abs().double()).sum())
    left, right = float((grad.double() * v.double()).sum()), float((y.double() * dy.double()).sum())
    assert abs(left - right) <= 2 * 2.0 ** -19 * mag


def test_runs_on_the_given_stream(eg):
    import torch
    ids = torch.from_numpy(make_ids(9000, 2, 700, "skewed", 4)).cuda()
    dy = make_dy(9000, 2, 64, "bf16", False, 4).cuda()
    want = eg.engram_embed_grad(ids, dy, 700)
    s, late = torch.cuda.Stream(), torch.zeros_like(dy)
    grad = torch.empty_like(want)
    ws = torch.empty(eg.engram_embed_grad_workspace_bytes(9000, 2, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(dy, non_blocking=True)
    eg.engram_embed_grad(ids, late, 700, grad=grad, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(grad, want)


@pytest.mark.parametrize("T,R", [(6143, 1), (1536, 4), (6145, 1), (1229, 5), (622591, 1), (207532, 3)])
@pytest.mark.parametrize("kind", ["skewed", "uniform"])
def test_list_lengths_where_the_sort_changes(eg, T, R, kind):
    import torch
    D, rows = 8, 200003
    ids, dy = make_ids(T, R, rows, kind, seed=T), make_dy(T, R, D, "f32", False, seed=T)
    uniq, ref, bound = reference(ids, dy, rows, 0.37, False)
    ci, cd = torch.from_numpy(ids).cuda(), dy.cuda()
    grad = eg.engram_embed_grad(ci, cd, rows, scale=0.37)
    row_ids, grads, count = eg.engram_embed_grad_rows(ci, cd, rows, scale=0.37)
    n = int(count)
    got_ids = row_ids.cpu().numpy()
    assert n == len(uniq) and (got_ids[:n] == uniq).all() and (got_ids[n:] == -1).all()
    close(grads[:n].double().cpu().numpy(), ref, bound, "f32")
    assert torch.equal(grads[:n], grad[torch.from_numpy(uniq).cuda()])
    grad[torch.from_numpy(uniq).cuda()] = 0
    assert not grad.any()
