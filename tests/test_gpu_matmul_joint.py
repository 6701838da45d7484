"""The gradient's two products in one launch: CTAs walk from the tiles of one into those of the other
while their warps are at different tiles, so the second's buffers must not lie where the first's
still are.  Outputs of different types and an added db give the two products buffers of different
sizes; a share of a tile that is empty (widths that no part of the warps divides, rows past a ragged
edge) lets warps run ahead of one another.

Each output is compared with the fp64 product, with the tolerance of a product in tests/
test_gpu_matmul.py: (length/16 + 16) 2^-22 of sum |dz b| for the sums and half a step of its type
(an output that another warp's values fell into is off by the size of a value), and a db that is
added to half a step of the sum more, 2^-24 of the old value with it; every repetition has the bits
of the first."""
import pytest

pytestmark = pytest.mark.gpu
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def eg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_memory_gb300 as eg
    return eg


# Pairs and single CTAs, the first product's tiles the longer ones and the second's; M under N and
# over it, edges that end inside a tile, sums in one accumulator and in segments.
SIZES = [(512, 4096, 6144), (320, 2048, 2048), (300, 1000, 1536), (1000, 200, 776), (2056, 520, 1160), (130, 2056, 4104),
         (4100, 2304, 512), (1100, 1104, 8200)]


@pytest.mark.parametrize("da,db,accumulate", [("bf16", "f32", True), ("bf16", "f32", False), ("f32", "bf16", True),
                                              ("bf16", "bf16", True), ("f32", "f32", True)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_two_products_in_one_launch(eg, M, N, K, da, db, accumulate):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    dy, a, b = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((M, N), (M, K), (N, K)))
    old = torch.randn(N, K, generator=g, device="cuda").to(dt[db])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return eg.engram_matmul_grad(dy, a, b, accumulate=accumulate, da_dtype=dt[da], db_dtype=dt[db],
                                     db=old.clone() if accumulate else None, status=status)[:2]
    first = call()
    y, added = dy.double(), old.double() if accumulate else torch.zeros(1, device="cuda", dtype=torch.float64)
    for got, want, S, length, kind in (
            (first[0], y @ b.double(), y.abs() @ b.double().abs(), N, da),
            (first[1], y.t() @ a.double() + added, y.t().abs() @ a.double().abs(), M, db)):
        slack = (length / 16 + 16) * 2.0 ** -22 * S + HALF_STEP[kind] * want.abs()
        if got is first[1]:
            slack = slack + 2.0 ** -23 * added.abs()
        assert ((got.double() - want).abs() <= slack).all()
    for _ in range(20):
        assert all(torch.equal(x, w) for x, w in zip(call(), first))
    assert eg.engram_read_status(status) == (eg.OK, 0)
