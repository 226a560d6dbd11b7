"""Products in each of their kernels: which one ran, and what each has of its
own."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from kernel_nodes import kernels_of  # noqa: E402
from matrices_harness import Codes  # noqa: E402
from oracle import matrices as O  # noqa: E402
from test_matrix8_gpu import PAIRS, check_product  # noqa: E402


def kernel_of(m, n, k, dtype=torch.float32):
    """(rows of a per tile or "pair", CTAs that share a tile's k) of the kernel that a product of this size takes."""
    a, b, d = Codes(m, k), Codes(n, k), torch.zeros(m, n, dtype=dtype, device="cuda")
    dopt.dopt_matrix8_multiply(a.m, b.m, d, stream=torch.cuda.current_stream())
    (name, ctas, _), = kernels_of(lambda s: dopt.dopt_matrix8_multiply(a.m, b.m, d, stream=s))
    if "matrix8_multiply_pair" in name:
        return "pair", 1
    for rows in (16, 32, 64, 128):
        for split in (0, 1):
            if f"matrix8_multiplyILi{rows}ELb{split}E" in name:
                assert split == (ctas > 1)
                return rows, ctas
    raise AssertionError(name)


# Few columns of the last tile, not by four: of a warp some lanes store four, one some, the others none.
SPLITS = {(16, 2): (10, 16898, 3000), (16, 4): (10, 2435, 4096), (16, 8): (10, 130, 4096),
          (32, 2): (30, 16899, 3000), (32, 4): (30, 4994, 2048), (32, 8): (20, 129, 4096),
          (64, 2): (60, 16897, 4000), (64, 4): (60, 4993, 3000), (64, 8): (60, 131, 4096),
          (128, 2): (100, 5890, 5000), (128, 4): (100, 2945, 4096), (128, 8): (100, 257, 4096)}


@pytest.mark.parametrize("which", sorted(SPLITS))
def test_parts_of_k_of_partial_columns(which):
    """A cluster adds up its CTAs' parts of k; lanes of a warp that store differently meet again at its barriers."""
    m, n, k = SPLITS[which]
    assert kernel_of(m, n, k) == which
    outputs = [("f32", False, 0), ("bf16", False, 3), ("f16", True, 1)]
    for dtype, add, pad in outputs if n < 1000 else [outputs[m % 3]]:
        check_product(m, n, k, dtype, add=add, pad=pad)


@pytest.mark.parametrize("rows", [1, 3])
def test_product_of_nothing_into_far_rows(rows):
    """Without columns the sums are 0, also in rows more than 2^31 bytes apart, and only there."""
    ld = 2**30 + 512
    whole = torch.ones((rows - 1) * ld + 64, dtype=torch.bfloat16, device="cuda")
    d = whole.as_strided((rows, 5), (ld, 1))
    a, b = Codes(rows, 0), Codes(5, 0)
    for add in (True, False):
        dopt.dopt_matrix8_multiply(a.m, b.m, d, accumulate=add, stream=torch.cuda.current_stream())
        assert bool((d == int(add)).all())
        d.fill_(1)
        assert bool((whole == 1).all())
    # nothing is left for the next call to find
    check_product(rows, 5, 40, "bf16")


@pytest.mark.parametrize("which,sizes", [(("pair", 1), PAIRS[0]), (("pair", 1), PAIRS[1]), (("pair", 1), (16384, 11008, 4096)),
                                         ((16, 1), (3, 39000, 200)), ((32, 1), (30, 39000, 200)), ((64, 1), (60, 39000, 200)),
                                         ((128, 1), (100, 39000, 200)), ((128, 1), (2049, 2500, 600)), ((128, 1), (700, 11000, 384))])
def test_the_kernel_that_other_tests_are_meant_for(which, sizes):
    """Sizes by which test_matrix8_gpu.py reaches each kernel, and the one that a large product takes."""
    for dtype in (torch.float32, torch.bfloat16):
        assert kernel_of(*sizes, dtype) == which


# Sums along k that have no sign: what the matrix unit loses adds up.  fp32 results are summed there over 4096 of k at
# most, so a term passes 32 additions in its step and 128 from step to step, each off by at most one last place (2 U),
# and then additions to nearest (U): of 65 parts, and of a cluster's eight CTAs.  Summed there whole, 262144 of k and more
# are off by 5e-5 (as measured 3.1e-6 at 16384, in proportion) to 1.7e-4 (if every step cuts off what does not fit).
K = 262144 + 200
PARTS_BOUND = 2 * O.U * (32 + 128) + O.U * (65 + 8)


@pytest.mark.parametrize("which,m,n", [((16, 8), 3, 200), ((128, 8), 100, 300), ((128, 1), 100, 9800), (("pair", 1), 1000, 3900)])
def test_sums_of_one_sign_along_a_long_k(which, m, n):
    gen = torch.Generator("cuda").manual_seed(m + n)
    a, b = (torch.randint(1, 64, (rows, -(-K // 16) * 16), generator=gen, device="cuda", dtype=torch.uint8)[:, :K] for rows in (m, n))
    ma, mb = (dopt.Matrix8(x, torch.full((dopt.dopt_matrix8_scale_bytes(*x.shape),), 127, dtype=torch.uint8, device="cuda")) for x in (a, b))
    at = torch.tensor(sorted({0, 1, m // 2, m - 1}), device="cuda")

    def numbers(codes):
        return codes.contiguous().view(torch.float8_e4m3fn).double()

    want = torch.cat([numbers(a[at]) @ numbers(b[c:c + 500]).t() for c in range(0, n, 500)], 1)
    d = torch.zeros(m, n, device="cuda")
    dopt.dopt_matrix8_multiply(ma, mb, d, stream=torch.cuda.current_stream())
    assert float((d[at].double() / want - 1).abs().max()) < PARTS_BOUND < 2.4e-5
    assert kernel_of(m, n, K) == which
    # 16-bit results: as many as 131072 of k there, so two parts and more here
    d = d.bfloat16()
    dopt.dopt_matrix8_multiply(ma, mb, d, stream=torch.cuda.current_stream())
    assert kernel_of(m, n, K, torch.bfloat16) == which
    assert float((d[at].double() / want - 1).abs().max()) < O.EPS["bf16"] + 2 * O.U * (32 + K / 32 + 8)
