"""The README's lines for products of 8-bit matrices run as they stand."""

import os
import textwrap

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from oracle import matrices as O  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_lines():
    text = open(os.path.join(ROOT, "README.md")).read()
    lines = text[text.index("    def matrix8(rows, cols):"):].split("\n")
    end = next(i for i, line in enumerate(lines) if line and not line.startswith("    "))
    return textwrap.dedent("\n".join(lines[:end]))


def test_readme_products():
    torch.manual_seed(1)
    T, D, F = 70, 200, 130
    weight, x = torch.randn(F, D, device="cuda") * 0.05, torch.randn(T, D, device="cuda").bfloat16()
    dy, grad = torch.randn(T, F, device="cuda").bfloat16(), torch.randn(F, D, device="cuda")
    y, dx, before = torch.empty_like(dy), torch.empty_like(x), grad.clone()
    exec(readme_lines(), dict(torch=torch, dopt=dopt, T=T, D=D, F=F, weight=weight, x=x, dy=dy, grad=grad, y=y, dx=dx))

    def rounded(t, square=False):
        v = t.double().cpu().numpy()
        return O.rounded(v, O.scales(v, square))

    for got, a, b, old, dtype in ((y, rounded(x), rounded(weight, True), 0, "bf16"), (dx, rounded(dy), rounded(weight.t(), True), 0, "bf16"),
                                  (grad, rounded(dy.t()), rounded(x.t()), before.double().cpu().numpy(), "f32")):
        want, bound = O.product(a, b)
        assert O.near(got.double().cpu().numpy(), want + old, bound + O.U * abs(want + old), dtype).all()
