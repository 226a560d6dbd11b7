"""Arrays that lie between each other without sharing an element: outputs in
one buffer, as columns of it or one after another."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402

ROWS, COLS = 50, 264


def runs(place):
    """h and y, dh and dx, and a dropout's y, in memory that place(k, i) gives: call k's i-th output."""
    gen = torch.Generator("cuda").manual_seed(1)
    x, res, dy = (torch.randn(ROWS, COLS, generator=gen, device="cuda").bfloat16() for _ in range(3))
    gain, rstd, drop, s = torch.ones(COLS, device="cuda"), torch.empty(ROWS, device="cuda"), dopt.Dropout(0.1, 5), torch.cuda.current_stream()
    out = [place(k, i) for k in range(2) for i in range(2)]
    dopt.dopt_rms_norm(dopt.RmsNormArgs(x, gain, 1e-6, residual=res, dropout=drop, h=out[0], y=out[1], rstd=rstd), stream=s)
    dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(dy, out[0], gain, rstd, out[2], dres=res, dropout=drop, dx=out[3]), stream=s)
    both = torch.cat([x.flatten(), torch.zeros(ROWS * COLS, device="cuda", dtype=x.dtype)])
    dopt.dopt_dropout(dopt.DropoutArgs(both[: ROWS * COLS], both[ROWS * COLS:], drop), stream=s)
    return [t.clone() for t in out] + [both]


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_outputs_between_each_other(pad):
    apart = runs(lambda k, i: torch.zeros(ROWS, COLS + pad, device="cuda", dtype=torch.bfloat16)[:, :COLS])
    wide = [torch.zeros(ROWS, 2 * (COLS + pad), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    beside = runs(lambda k, i: wide[k][:, i * (COLS + pad):][:, :COLS])
    tall = [torch.zeros(2 * ROWS, COLS + pad, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    below = runs(lambda k, i: tall[k][i * ROWS:][:ROWS, :COLS])
    for a, b, c in zip(apart, beside, below):
        assert torch.equal(a, b) and torch.equal(a, c)
