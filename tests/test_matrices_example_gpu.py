"""The example with 8-bit matrices runs, and its gradients are those of its
formulas, computed by torch in 64 bits through the same dropout masks from
the rounded matrices that each product had."""

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from oracle import matrices as O  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import tensor_list_step as E  # noqa: E402


@pytest.mark.parametrize("moments", [8, 32])
def test_the_example_runs(moments):
    losses, norm, applied = E.train(moments=moments, steps=12, matrices=8, layers=3, batch=300, d=136)
    assert applied == 12 and np.isfinite(losses).all() and np.isfinite(norm)


def rounded(x, square=False):
    x = x.detach().double().cpu().numpy()
    return torch.from_numpy(O.rounded(x, O.scales(x, square)))


def test_product_gradients():
    """Against the products of the matrices as they are packed, within fp32's bound and the outputs' roundings."""
    torch.manual_seed(1)
    x = torch.randn(70, 136, device="cuda").bfloat16().requires_grad_()
    w = (torch.randn(200, 136, device="cuda") * 0.05).bfloat16().requires_grad_()
    dy = torch.randn(70, 200, device="cuda").bfloat16()
    w8, w8_t = E.matrix8(200, 136), E.matrix8(136, 200)
    dopt.dopt_matrix8_pack(dopt.MatrixList([dict(values=w.detach(), block=dopt.BLOCK_SQUARE, out=w8, out_t=w8_t)]), stream=E.stream())
    y = E.Product8.apply(x, w, w8, w8_t)
    y.backward(dy)
    for got, a, b in ((y, rounded(x), rounded(w, True)), (x.grad, rounded(dy), rounded(w.t(), True)),
                      (w.grad, rounded(dy.t()), rounded(x.t()))):
        want, bound = O.product(a.numpy(), b.numpy())
        assert O.near(got.detach().double().cpu().numpy(), want, bound, "bf16").all()


def test_norm_gradients():
    """Against torch's gradients of the formula in fp64, and with the mask that a dropout of ones shows.  The norm's
    outputs and gradients are bf16 of values within a few fp32 ulps: 2^-8 of each; h's rounding to bf16, which the
    formula sees too, is repeated here."""
    torch.manual_seed(2)
    rows, cols = 60, 136
    x, branch = (torch.randn(rows, cols, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    gain = (1 + 0.1 * torch.randn(cols, device="cuda")).requires_grad_()
    dh, dy = (torch.randn(rows, cols, device="cuda").bfloat16() for _ in range(2))
    drop = dopt.Dropout(0.25, 7, site=3, step=5)
    h, y = E.Norm8.apply(x, branch, gain, drop)
    torch.autograd.backward((h, y), (dh, dy))
    mask = torch.empty(rows, cols, device="cuda")
    dopt.dopt_dropout(dopt.DropoutArgs(torch.ones_like(mask), mask, drop), stream=E.stream())
    leaf = h.detach().double().requires_grad_()
    g = gain.detach().double().requires_grad_()
    norm = leaf * torch.rsqrt((leaf * leaf).mean(1, keepdim=True) + 1e-6) * g
    torch.autograd.backward((leaf, norm), (dh.double(), dy.double()))
    exact_h = branch.detach().double() * mask.double() + x.detach().double()
    half = 2.0**-8

    def near(got, want, scale):
        # a few ulps of fp32 of the terms that cancel (scale), and half a step of bf16
        got, want = got.detach().double(), want.detach()
        assert bool(((got - want).abs() <= half * want.abs() + 64 * 2.0**-24 * scale + 2.0**-133).all())

    near(h, exact_h, exact_h.abs())
    near(y, norm, norm.abs())
    terms = leaf.grad.abs() + dh.double().abs() + (dy.double() * g).abs() + norm.abs()
    near(x.grad, leaf.grad, terms.amax(1, keepdim=True))
    near(branch.grad, leaf.grad * mask.double(), 2 * terms.amax(1, keepdim=True))
    assert bool(((gain.grad.double() - g.grad).abs() <= 100 * 2.0**-24 * (dy.double() * norm / g).abs().sum(0)).all())


def test_losses_gradients_by_differences():
    """The whole model's gradient in one direction against the difference of its loss along it.  In 8 bits the loss is
    a staircase, so that the model is compared with itself: without a matrix's rounding (weights and activations that
    are e4m3 numbers of one size) nothing of it is left but the formula."""
    torch.manual_seed(3)
    x = torch.randint(-8, 9, (64, 128), device="cuda").float().requires_grad_()
    w = torch.randint(-8, 9, (96, 128), device="cuda").float().requires_grad_()
    w8, w8_t = E.matrix8(96, 128), E.matrix8(128, 96)

    def pack(weight):
        dopt.dopt_matrix8_pack(dopt.MatrixList([dict(values=weight.detach(), block=dopt.BLOCK_SQUARE, out=w8, out_t=w8_t)]),
                               stream=E.stream())

    def product(a, b):
        pack(b)
        return E.Product8.apply(a, b, w8, w8_t)

    dy = torch.randint(-8, 9, (64, 96), device="cuda").float()
    (product(x, w) * dy).sum().backward()
    step_x, step_w = (torch.randint(-4, 5, t.shape, device="cuda").float() for t in (x, w))
    with torch.no_grad():
        # numbers up to 12 and down to -12 are e4m3's own, and the product is linear in each: differences are exact
        up, down = product(x + step_x, w), product(x - step_x, w)
        assert float(((up - down) * dy).sum()) / 2 == float((x.grad * step_x).sum())
        up, down = product(x, w + step_w), product(x, w - step_w)
        assert float(((up - down) * dy).sum()) / 2 == float((w.grad * step_w).sum())
