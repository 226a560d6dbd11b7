"""Dropout with a residual, bit for bit: the product and the sum are each
rounded in fp32, and the sum then to the arrays' type."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from matrices_harness import TORCH  # noqa: E402
from oracle import matrices as O  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,offset", [(5000, 0), (5003, 1)])
def test_each_operation_rounds_once(n, offset, dtype):
    gen = torch.Generator("cuda").manual_seed(n)
    x, res, y = (torch.randn(n + offset, generator=gen, device="cuda").to(TORCH[dtype])[offset:] for _ in range(3))
    dopt.dopt_dropout(dopt.DropoutArgs(x, y, dopt.Dropout(0.3, 7, site=2, step=5), residual=res), stream=torch.cuda.current_stream())
    h, rstd = torch.empty(1, n, dtype=x.dtype, device="cuda"), torch.empty(1, device="cuda")
    dopt.dopt_rms_norm(dopt.RmsNormArgs(x[None], torch.ones(n, device="cuda"), 1e-6, residual=res[None], h=h, y=torch.empty_like(h), rstd=rstd,
                                        dropout=dopt.Dropout(0.3, 7, site=2, step=5)), stream=torch.cuda.current_stream())
    drop = O.threshold(0.3)
    gone = O.random16(np.arange(n), 7, 2, 5) < drop
    keep = np.float32(65536 / (65536 - drop))
    a, b = x.float().cpu().numpy(), res.float().cpu().numpy()
    want = np.where(gone, np.float32(0), a * keep) + b
    assert want.dtype == np.float32
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(TORCH[dtype])) and torch.equal(h[0], y)
    # which is not the sum of the exact product, rounded once
    once = np.where(gone, 0.0, a.astype(np.float64) * np.float64(keep)) + b
    assert dtype != "f32" or (once.astype(np.float32) != want).any()
