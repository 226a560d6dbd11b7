"""8-bit matrices and their products on the GPU against the 64-bit
restatement: every code and scale byte of pack, every value of unpack, and
products within the bound of fp32 sums."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from matrices_harness import Codes, Rows, empty, numbers, stored  # noqa: E402
from oracle import matrices as O  # noqa: E402

SIZES = [(1, 1), (1, 300), (3, 128), (128, 128), (127, 129), (129, 127), (257, 640), (300, 1030), (16, 2048)]


def stream():
    return torch.cuda.current_stream()


def pack(x, dtype, square=False, straight=True, turned=True, pad=0, offset=0):
    src = Rows(x, dtype, pad, offset)
    rows, cols = x.shape
    out = Codes(rows, cols, 1) if straight else None
    out_t = Codes(cols, rows, 2) if turned else None
    e = dict(values=src.view, block=dopt.BLOCK_SQUARE if square else dopt.BLOCK_ROW)
    if straight:
        e["out"] = out.m
    if turned:
        e["out_t"] = out_t.m
    dopt.dopt_matrix8_pack(dopt.MatrixList([e]), stream=stream())
    torch.cuda.synchronize()
    assert src.guards_intact()
    return out, out_t


def check_packed(m, x, square):
    s = O.scales(x, square)
    assert np.array_equal(m.scale_bytes(), s)
    assert np.array_equal(m.numpy(), O.rounded(x, s), equal_nan=True)
    assert m.guards_intact()


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack(rows, cols, dtype, square):
    x = stored(numbers(rows, cols, rows * 7 + cols), dtype)
    for straight, turned, pad, offset in ((True, True, 0, 0), (True, False, 3, 1), (False, True, 8, 4)):
        out, out_t = pack(x, dtype, square, straight, turned, pad, offset)
        if straight:
            check_packed(out, x, square)
        if turned:
            check_packed(out_t, x.T.copy(), square)


@pytest.mark.parametrize("square", [False, True])
def test_pack_extremes(square):
    """Zeros, the borders of the scale, subnormals, infinities and NaN, the type's largest values."""
    x = stored(numbers(300, 400, 5), "f32")
    x[:140, :130] = 0
    x[200, 3], x[201, 300], x[299, 399] = np.inf, np.nan, -np.inf
    x[140:142, 140:300] = 2.0**-140
    x[150, 260:270] = 3.4e38
    x[160, 260:384] = 2.0**-126 * 448
    for k, top in enumerate((448.0, 448.1, 480.0, 480.1, 1.75, 1.76)):
        x[170 + k, 256:384] = np.linspace(-1, 1, 128) * top
    x = stored(x, "f32")
    out, out_t = pack(x, "f32", square)
    with np.errstate(invalid="ignore"):
        check_packed(out, x, square)
        check_packed(out_t, x.T.copy(), square)
    # a NaN block's codes are 0
    bad = O.per_column(out.scale_bytes(), 400) == 255
    assert bad.any() and (out.codes.cpu().numpy()[bad] == 0).all()


def test_pack_a_list():
    """More matrices than a launch's table holds, of every type, an empty one among them, and one launch for few."""
    rng = np.random.default_rng(3)
    xs = [stored(numbers(int(r), int(c), k), d) for k, (r, c, d) in enumerate(
        zip(rng.integers(1, 200, 330), rng.integers(1, 300, 330), ["f32"] * 310 + ["bf16", "f16"] * 10))]
    src = [Rows(x, "f32" if k < 310 else ("bf16", "f16")[k % 2]) for k, x in enumerate(xs)]
    out = [(Codes(*x.shape), Codes(*x.T.shape)) for x in xs]
    entries = [dict(values=s.view, out=a.m, out_t=b.m, block=k % 2) for k, (s, (a, b)) in enumerate(zip(src, out))]
    entries.insert(5, dict(values=torch.zeros(0, 7, device="cuda"), out=dopt.Matrix8(
        torch.zeros(0, 16, dtype=torch.uint8, device="cuda")[:, :7], torch.zeros(0, dtype=torch.uint8, device="cuda"))))
    before = dopt.dopt_kernel_launches()
    dopt.dopt_matrix8_pack(dopt.MatrixList(entries), stream=stream())
    assert dopt.dopt_kernel_launches() - before == 4
    for k, (x, (a, b)) in enumerate(zip(xs, out)):
        check_packed(a, x, k % 2)
        check_packed(b, x.T.copy(), k % 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_unpack(rows, cols, dtype):
    m = Codes(rows, cols, 1)
    rng = np.random.default_rng(rows + cols)
    c = rng.integers(0, 256, (rows, cols))
    c[(c & 127) == 127] = 3  # e4m3's NaN codes are never stored
    m.codes.copy_(torch.from_numpy(c.astype(np.uint8)))
    s = rng.integers(8, 247, (rows, O.blocks_of(cols)))
    s[rng.random(s.shape) < 0.1] = 255
    m.set_scales(s)
    for pad, offset in ((0, 0), (5, 1)):
        out = empty(rows, cols, dtype, pad, offset)
        dopt.dopt_matrix8_unpack(dopt.MatrixList([dict(values=out.view, out=m.m)]), stream=stream())
        assert np.array_equal(out.numpy(), O.values(c, s), equal_nan=True)
        assert out.guards_intact()


# ----------------------------------------------------------------- products --

def multiply(a, b, dtype, add=None, pad=0, offset=0):
    d = empty(a.rows, b.rows, dtype, pad, offset) if add is None else Rows(add, dtype, pad, offset)
    dopt.dopt_matrix8_multiply(a.m, b.m, d.view, accumulate=add is not None, stream=stream())
    got = d.numpy()
    assert d.guards_intact()
    return got


def check_product(m, n, k, dtype, square=False, add=False, pad=0, offset=0, seed=0):
    a, b = Codes(m, k), Codes(n, k, 1)
    av, bv = a.fill(numbers(m, k, seed + m), False), b.fill(numbers(n, k, seed + n + 1), square)
    want, bound = O.product(av, bv)
    old = stored(numbers(m, n, seed + 2), dtype) if add else None
    if add:
        want = want + old
        bound = bound + O.U * np.abs(want)
    got = multiply(a, b, dtype, old, pad, offset)
    ok = O.near(got, want, bound, dtype)
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4])


@pytest.mark.parametrize("m", [1, 15, 16, 17, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(128, 128), (1, 1), (130, 515), (255, 2048), (384, 1000)])
def test_product(m, n, k):
    check_product(m, n, k, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (64, 8)])
def test_product_outputs(dtype, add, pad, offset):
    for m, n, k in ((5, 200, 700), (140, 200, 700), (100, 129, 130)):
        check_product(m, n, k, dtype, square=True, add=add, pad=pad, offset=offset)


@pytest.mark.parametrize("m,n,k", [(2049, 2500, 600), (5000, 2000, 129), (700, 11000, 384), (257, 20000, 130)])
def test_product_many_tiles(m, n, k):
    """More tiles than CTAs: the ring and the sums go on from tile to tile."""
    check_product(m, n, k, "bf16")


# Tiles of two SMs are for products whose tiles fill the SMs that way and whose k is long: one tile for each pair of
# them, and several.
PAIRS = [(1000, 3900, 3100), (2300, 4300, 5000)]


@pytest.mark.parametrize("m,n,k", [(40, 300, 4096), (40, 300, 20000), (100, 300, 40000), (1500, 1000, 4096), (1500, 1000, 4300),
                                   (2500, 2300, 4097)] + PAIRS)
@pytest.mark.parametrize("dtype,add", [("f32", False), ("f32", True), ("bf16", False)])
def test_product_long_sums(m, n, k, dtype, add):
    """Sums that are added up in parts, in every kernel: one tile's, a cluster's and a pair's."""
    check_product(m, n, k, dtype, add=add)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_product_of_pairs_added(dtype):
    """Tiles of two SMs added to what is there, odd rows of d."""
    check_product(*PAIRS[0], dtype, add=True, pad=3, offset=1)


@pytest.mark.parametrize("m", [50, 300])
def test_product_with_itself(m):
    a = Codes(m, 900)
    av = a.fill(numbers(m, 900, m))
    want, bound = O.product(av, av)
    got = multiply(a, a, "f32")
    assert O.near(got, want, bound, "f32").all()


@pytest.mark.parametrize("m", [3, 30, 60, 100])
def test_product_more_tiles_than_fit(m):
    """Few rows of a and so many of b that nothing is split."""
    check_product(m, 39000, 200, "bf16")


@pytest.mark.parametrize("m,n", [(7, 200), (100, 200), (300, 200), (1000, 3900)])
def test_product_is_exact_on_small_integers(m, n):
    """Whole numbers whose sums fit 24 bits: every product and sum is exact, in any order, in fp32."""
    k = 4096
    rng = np.random.default_rng(m)
    a, b = Codes(m, k), Codes(n, k)
    av, bv = rng.integers(-15, 16, (m, k)).astype(float), rng.integers(-15, 16, (n, k)).astype(float)
    for x, v in ((a, av), (b, bv)):
        x.codes.copy_(torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8))
        x.set_scales(np.full((x.rows, O.blocks_of(k)), 127))
    assert np.array_equal(multiply(a, b, "f32"), av @ bv.T)


def test_product_scales_of_every_block():
    """One number per block, each with a scale of its own: a wrong row, block or byte shows at once."""
    m, n, k = 300, 260, 128 * 9
    a, b = Codes(m, k), Codes(n, k)
    rng = np.random.default_rng(1)
    for x in (a, b):
        c = np.zeros((x.rows, k))
        for blk in range(9):
            c[np.arange(x.rows), blk * 128 + (np.arange(x.rows) if x is a else rng.integers(0, 128, x.rows)) % 128] = 1
        c[:, ::128] = 1
        x.codes.copy_(torch.from_numpy(c).to(torch.float8_e4m3fn).view(torch.uint8))
        x.set_scales(rng.integers(110, 144, (x.rows, 9)))
        x.v = x.numpy()
    want, bound = O.product(a.v, b.v)
    assert O.near(multiply(a, b, "f32"), want, bound, "f32").all()


@pytest.mark.parametrize("m,n,k", [(20, 300, 700), (200, 300, 700), (1000, 300, 700), PAIRS[0]])
def test_product_nan_blocks(m, n, k):
    """A block that reads as NaN makes its row (of a) or column (of b) NaN, and nothing else."""
    a, b = Codes(m, k), Codes(n, k)
    av, bv = a.fill(numbers(m, k, 1)), b.fill(numbers(n, k, 2))
    sa, sb = a.scale_bytes(), b.scale_bytes()
    sa[m // 2, 5] = 255
    sb[129, 2] = 255
    a.set_scales(sa)
    b.set_scales(sb)
    got = multiply(a, b, "f32")
    want, bound = O.product(av, bv)
    bad = np.zeros((m, n), bool)
    bad[m // 2], bad[:, 129] = True, True
    assert np.isnan(got[bad]).all()
    assert O.near(got, want, bound, "f32")[~bad].all()


def test_product_extremes():
    """Scales at both ends: sums that are infinite, and terms too small for fp32."""
    m, n, k = 130, 140, 256
    a, b = Codes(m, k), Codes(n, k)
    a.fill(np.abs(numbers(m, k, 1)) + 0.1)
    b.fill(np.abs(numbers(n, k, 2)) + 0.1)
    for s, want in ((240, np.inf), (20, 0.0)):
        a.set_scales(np.full((m, 2), s))
        b.set_scales(np.full((n, 2), s))
        assert (multiply(a, b, "f32") == want).all()


def test_product_of_nothing():
    a, b = Codes(5, 0), Codes(7, 0)
    assert (multiply(a, b, "bf16", pad=3) == 0).all()
    old = stored(numbers(5, 7, 1), "f32")
    assert np.array_equal(multiply(a, b, "f32", old), old)
    d = torch.zeros(0, 7, device="cuda")
    dopt.dopt_matrix8_multiply(Codes(0, 30).m, Codes(7, 30).m, d, stream=stream())


@pytest.mark.parametrize("m", [3, 200])
def test_far_rows(m):
    """Rows more than 2^31 bytes and elements apart, of the operands and of d."""
    n, k = 5, 200
    if m > 3:
        a = Codes(m, k)
        av = a.fill(numbers(m, k, 1))
        whole = torch.zeros(4 * 2**30 + 2**20, dtype=torch.uint8, device="cuda")
        b = Codes(n, k)
        bv = b.fill(numbers(n, k, 2))
        far = whole.as_strided((n, k), (2**30, 1))
        far.copy_(b.codes)
        d = torch.zeros(m, n, device="cuda")
        dopt.dopt_matrix8_multiply(a.m, dopt.Matrix8(far, b.scales), d, stream=stream())
        d = d.double().cpu().numpy()
    else:
        a, b = Codes(m, k), Codes(n, k)
        av, bv = a.fill(numbers(m, k, 1)), b.fill(numbers(n, k, 2))
        whole = torch.zeros(2 * (2**30 + 512) + 64, dtype=torch.bfloat16, device="cuda")
        view = whole.as_strided((m, n), (2**30 + 512, 1))
        dopt.dopt_matrix8_multiply(a.m, b.m, view, stream=stream())
        d = view.double().cpu().numpy()
        view.zero_()
        assert not bool(whole.any())
        x = stored(numbers(m, 300, 3), "bf16")
        wide = whole.as_strided((m, 40), (2**30 + 512, 1))
        wide.copy_(torch.from_numpy(x[:, :40]))
        out = Codes(m, 40)
        dopt.dopt_matrix8_pack(dopt.MatrixList([dict(values=wide, out=out.m)]), stream=stream())
        check_packed(out, x[:, :40].copy(), False)
    want, bound = O.product(av, bv)
    assert O.near(d, want, bound, "f32" if m > 3 else "bf16").all()


def test_two_products_at_once():
    """On two streams, with nothing between them."""
    cases = []
    for j, (m, n, k) in enumerate([(60, 500, 3000), (300, 500, 3000), PAIRS[0]]):
        a, b = Codes(m, k), Codes(n, k)
        want = O.product(a.fill(numbers(m, k, j)), b.fill(numbers(n, k, j + 5)))
        cases.append((a, b, torch.zeros(m, n, device="cuda"), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, b, d, _, s in cases:
            dopt.dopt_matrix8_multiply(a.m, b.m, d, stream=s)
    torch.cuda.synchronize()
    for _, _, d, (want, bound), _ in cases:
        assert O.near(d.double().cpu().numpy(), want, bound, "f32").all()


@pytest.mark.parametrize("m,n,k", [(40, 700, 5000), (400, 700, 5000), PAIRS[0]])
def test_product_is_the_same_every_time(m, n, k):
    a, b = Codes(m, k), Codes(n, k)
    a.fill(numbers(m, k, 1))
    b.fill(numbers(n, k, 2))
    first = multiply(a, b, "f32")
    for _ in range(5):
        assert np.array_equal(multiply(a, b, "f32"), first)
