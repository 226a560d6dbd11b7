"""The RMS norm of rows whose squares leave fp32's range at its lower end, and
of an eps that does, against the 64-bit restatement."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from matrices_harness import check_codes, numbers, stored  # noqa: E402
from oracle import matrices as O  # noqa: E402
from test_norm_dropout_gpu import assert_near, run_norm  # noqa: E402

# a warp has a row, or a CTA has; on the vector grid and off it
COLS = [200, 201, 704, 701, 2048, 4100, 16384]


def small_rows(cols, dtype):
    """Rows of about 1 down to the smallest values that there are, and of one such value alone."""
    x = numbers(12, cols, cols, spread=0.5)
    for r, size in enumerate((1.0, 1e-10, 1e-14, 1e-16, 1e-18, 1e-20, 1e-21, 1e-22, 1e-24, 1e-30, 1e-38, 1e-40)):
        x[r] *= size
    one = np.zeros((2, cols))
    one[0, cols // 2] = {"f32": 2.0**-149, "bf16": 2.0**-133}[dtype]
    one[1, cols - 1] = -1e-23
    return stored(np.concatenate([x, one]), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_norm_of_small_rows(cols, dtype):
    """Without eps every row's values come out near 1, however small they are."""
    x = small_rows(cols, dtype)
    for eps in (0.0, 1e-45, 1e-36):
        gain, a, m, rstd = run_norm(x, dtype, eps=eps)
        x = a["x"].numpy()
        with np.errstate(over="ignore"):
            (r, dr), (y, dy) = O.norm(x, gain, eps)
        assert_near(rstd, r, dr, "f32")
        assert_near(a["y"].numpy(), y, dy, dtype)
        check_codes(m.numpy(), m.scale_bytes(), y, dy)


@pytest.mark.parametrize("cols", [200, 201, 704, 701])
def test_norm_with_an_eps_outside_fp32(cols):
    """An eps that fp32 holds as 0 or as infinity counts as it is given; rows of zeros are zeros with any eps but 0."""
    x = stored(numbers(4, cols, 3), "f32")
    x[1], x[2] = 0, x[2] * 1e-30
    x[2] = stored(x[2], "f32")
    for eps in (1e-60, 1e-300, 1e60, 3.5e38):
        gain, a, m, rstd = run_norm(x, "f32", eps=eps)
        with np.errstate(over="ignore"):
            (r, dr), (y, dy) = O.norm(x, gain, eps)
        assert_near(rstd, r, dr, "f32")
        assert_near(a["y"].numpy(), y, dy, "f32")
        check_codes(m.numpy(), m.scale_bytes(), y, dy)
    gain, a, m, rstd = run_norm(x, "f32", eps=0.0)
    assert np.isinf(rstd[1]) and np.isnan(a["y"].numpy()[1]).all() and (m.scale_bytes()[1] == 255).all()
    assert np.isfinite(a["y"].numpy()[[0, 2, 3]]).all()
