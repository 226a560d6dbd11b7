"""The step over a list of tensors at the ends of its ranges, against the
64-bit restatement: second moments in and below fp32's subnormals."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from oracle import tensors as O  # noqa: E402
from tests.tensors_harness import HP, Case, check_codes  # noqa: E402

TINY = 2.0**-150  # half a unit of an fp32 subnormal: a rounding's absolute error there


def check_small_step(case, step, hp, seed=0):
    """A step whose second moments may be subnormal: their absolute errors (dv) and eps's own count in the
    denominator, so the weight's bound comes from the ends of its numerator and denominator.  Roundings besides: as
    O.adamw counts them (18), and 8 for an approximate root and reciprocal, each within 2^-22."""
    after = case.values()
    for k, (a, b) in enumerate(zip(case.before, after)):
        m, v = case.moments(a, k)
        w = case.weights(a).astype(np.float64)
        (w1, m1, v1), (_, dm, dv) = O.adamw(w, a["grad"], m, v, hp, step)
        size, eps, corr = hp["lr"] / (1 - hp["beta1"]**step), hp["eps"], 1 - hp["beta2"]**step
        de = O.U * eps + TINY
        low = np.sqrt(np.maximum(v1 - dv, 0) / corr) + eps - de
        high = np.sqrt((v1 + dv) / corr) + eps + de
        u = m1 / (np.sqrt(v1 / corr) + eps)
        ends = [(m1 + s * dm) / d for s in (-1, 1) for d in (low, high)]
        off = np.max([np.abs(e - u) for e in ends], axis=0)
        most = np.max([np.abs(e) for e in ends], axis=0)
        bound = size * off + 1.01 * O.U * (3 * np.abs(w) + 26 * size * most) + (8 + size * 2.0**24) * TINY
        got = case.weights(b).astype(np.float64)
        ok = np.abs(got - w1) <= bound
        assert ok.all(), (k, "weight", np.flatnonzero(~ok)[:5], got[~ok][:3], w1[~ok][:3], bound[~ok][:3])
        if case.spec[k]["moments"] == 8:
            check_codes(b, m1, dm, v1, dv, O.rounding_fraction(case.spec[k]["numel"], k, step, seed), k)
        else:
            assert (np.abs(b["exp_avg"] - m1) <= dm).all() and (np.abs(b["exp_avg_sq"] - v1) <= dv).all(), k
    case.check_guards()
    case.before = after


@pytest.mark.parametrize("moments", [8, 32])
@pytest.mark.parametrize("eps", [1e-8, 1e-20, 1e-30, 1e-40])
@pytest.mark.parametrize("size", [1e-12, 1e-20, 1e-22])
def test_step_with_subnormal_second_moments(moments, eps, size):
    """From zero moments, grads whose squares are subnormal or vanish, and an eps that does not hide them."""
    hp = dict(HP, eps=eps)
    case = Case([dict(numel=n, param="f32", grad="f32", moments=moments, offset=offset, zero=zero)
                 for n in (256, 4099) for offset in (0, 1) for zero in (0.0, 0.3)], seed=17, grad_size=size)
    for a in case.arrays:
        for name in a:
            if name.startswith("exp_avg"):
                a[name].view.zero_()
    case.before = case.values()
    for step in (1, 2, 3):
        dopt.dopt_tensors_adam_step(case.list, hp, step)
        check_small_step(case, step, hp)


@pytest.mark.parametrize("moments", [8, 32])
@pytest.mark.parametrize("host_step", [0, -7])
def test_host_step_is_ignored_with_a_device_step(moments, host_step):
    """With the count on the device the host's is not looked at: the same bits whatever it is."""
    spec = [dict(numel=5000, param="bf16", grad="bf16", moments=moments)]
    one, two = Case(spec, seed=18), Case(spec, seed=18)
    ws = torch.zeros(dopt.dopt_tensors_workspace_bytes(1), dtype=torch.uint8, device="cuda")
    for case, step in ((one, 1), (two, host_step)):
        count = torch.tensor([4], dtype=torch.int64, device="cuda")
        dopt.dopt_tensors_step(case.list, HP, step, ws, ws.numel(), seed=3, d_step=count)
        assert count.item() == 5
    assert all(np.array_equal(x, y) for x, y in zip(one.values()[0].values(), two.values()[0].values()))
