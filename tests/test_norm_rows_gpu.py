"""The norm and its backward pass with more rows than the device holds at
once, of lengths on the vector grid, so that threads have several rows: the
loads of the next under this one, and the sums in turn."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from kernel_nodes import kernels_of  # noqa: E402
from matrices_harness import TORCH, Codes, numbers, stored  # noqa: E402
from test_norm_dropout_gpu import DROP, check_norm, run_backward  # noqa: E402


def values(rows, cols, seed, dtype):
    return stored(numbers(rows, cols, seed), dtype)


def rounds(call, rows, cols):
    """How many rows each thread has one after another, at least."""
    call(torch.cuda.current_stream())
    ctas = kernels_of(call)[0][2]
    return rows / (ctas * (8 if cols <= 512 else 1))  # a CTA has a row, or each of its eight warps


# A length for each kernel of each type, and rows for each to go round at least twice
LENGTHS = [(256, 9000), (512, 5500), (768, 3000), (2048, 2600), (4096, 1500), (8192, 1000), (16384, 400)]


@pytest.mark.parametrize("cols,rows,dtype", [(c, r, t) for c, r in LENGTHS for t in ("bf16", "f32")] + [(256, 9000, "f16"), (4096, 1500, "f16")])
def test_norm_of_many_rows(cols, rows, dtype):
    x, y, g = torch.ones(rows, cols, dtype=TORCH[dtype], device="cuda"), Codes(rows, cols), torch.ones(cols, device="cuda")
    args = dopt.RmsNormArgs(x, g, 1e-6, y8=y.m)
    assert rounds(lambda s: dopt.dopt_rms_norm(args, stream=s), rows, cols) > 2
    x = values(rows, cols, cols, dtype)
    check_norm(x, dtype, residual=values(rows, cols, cols + 1, dtype), drop=DROP, values=cols <= 512)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,rows", [(256, 7500), (512, 5200)])
def test_norm_backward_of_many_rows(cols, rows, dtype):
    x, g, r = torch.ones(rows, cols, dtype=TORCH[dtype], device="cuda"), torch.ones(cols, device="cuda"), torch.ones(rows, device="cuda")
    size = dopt.dopt_rms_norm_workspace_bytes(rows, cols)
    args = dopt.RmsNormBackwardArgs(x, x, g, r, x.clone(), dgain=g.clone(), workspace=torch.empty(size, dtype=torch.uint8, device="cuda"),
                                    workspace_bytes=size)
    assert rounds(lambda s: dopt.dopt_rms_norm_backward(args, stream=s), rows, cols) > 2
    h, dy, dres = (values(rows, cols, cols + k, dtype) for k in range(3))
    _, first = run_backward(h, dy, dtype, dres=dres, drop=DROP)
    _, again = run_backward(h, dy, dtype, dres=dres, drop=DROP)
    assert np.array_equal(first, again)


@pytest.mark.parametrize("rows", [1, 8, 64, 153, 608, 1216, 5000])
def test_norm_backward_leaves_no_sm_without_work(rows):
    """With dgain too: a CTA per row up to the SMs, and no fewer CTAs than those after that; never more partial sums than
    the workspace holds."""
    cols, sms = 1024, torch.cuda.get_device_properties(0).multi_processor_count
    h, dy = values(rows, cols, 1, "bf16"), values(rows, cols, 2, "bf16")
    run_backward(h, dy, "bf16", add=True)
    x, g, r = torch.ones(rows, cols, dtype=TORCH["bf16"], device="cuda"), torch.ones(cols, device="cuda"), torch.ones(rows, device="cuda")
    size = dopt.dopt_rms_norm_workspace_bytes(rows, cols)
    args = dopt.RmsNormBackwardArgs(x, x, g, r, x.clone(), dgain=g.clone(), workspace=torch.empty(size, dtype=torch.uint8, device="cuda"),
                                    workspace_bytes=size)
    dopt.dopt_rms_norm_backward(args, stream=torch.cuda.current_stream())
    ctas = kernels_of(lambda s: dopt.dopt_rms_norm_backward(args, stream=s))[0][2]
    assert min(rows, sms) <= ctas <= size // (4 * cols)
