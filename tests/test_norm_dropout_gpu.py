"""The RMS norm, its backward pass and dropout on the GPU against the 64-bit
restatement, within the bounds of fp32's roundings."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from matrices_harness import Codes, Rows, check_codes, empty, numbers, stored  # noqa: E402
from oracle import matrices as O  # noqa: E402

SIZES = [(1, 1), (5, 7), (3, 256), (9, 257), (40, 769), (17, 1024), (7, 1025), (6, 2048), (5, 2051), (4, 4096), (3, 4100),
         (3, 8192), (2, 8200), (2, 16384)]
DROP = dict(p=0.2, seed=77, site=5, t=13)
EPS = 1e-5


def stream():
    return torch.cuda.current_stream()


def dropout_of(d, d_step=None):
    return None if d is None else dopt.Dropout(d["p"], d["seed"], site=d["site"], step=d["t"], d_step=d_step)


def assert_near(got, want, bound, dtype):
    ok = O.near(got, want, bound, dtype)
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4])


# ------------------------------------------------------------------ dropout --

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,offset", [(1, 0), (7, 1), (8, 0), (2049, 0), (2047, 3), (100000, 8)])
def test_dropout(n, offset, dtype):
    x, res = stored(numbers(1, n, n), dtype), stored(numbers(1, n, n + 1), dtype)
    for r in (None, res):
        for p in (0.0, 0.2, 0.9):
            drop = dict(DROP, p=p)
            xs, rs, y = Rows(x, dtype, offset=offset), Rows(res, dtype, offset=offset), empty(1, n, dtype, offset=offset)
            args = dopt.DropoutArgs(xs.view[0], y.view[0], dropout_of(drop), residual=None if r is None else rs.view[0])
            dopt.dopt_dropout(args, stream=stream())
            want, bound = O.norm_input(x, r, drop)
            assert_near(y.numpy(), want, bound, dtype)
            assert y.guards_intact() and xs.guards_intact()
            dopt.dopt_dropout(dopt.DropoutArgs(xs.view[0], xs.view[0], dropout_of(drop), residual=None if r is None else rs.view[0]),
                              stream=stream())
            assert np.array_equal(xs.numpy(), y.numpy()) and xs.guards_intact()


def test_dropped_elements_are_zero_whatever_they_were():
    x = np.where(np.arange(5000) % 2, np.inf, np.nan)[None]
    xs, y = Rows(x, "f32"), empty(1, 5000, "f32")
    dopt.dopt_dropout(dopt.DropoutArgs(xs.view[0], y.view[0], dropout_of(DROP)), stream=stream())
    gone = O.random16(np.arange(5000), 77, 5, 13) < O.threshold(0.2)
    got = y.numpy()[0]
    assert (got[gone] == 0).all() and not np.isfinite(got[~gone]).any()


def test_dropout_backward_is_the_same_call():
    """The derivative of sum(dy * dropout(x)) by x, by torch, from the mask that the forward call showed."""
    n = 3001
    x, dy = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    shown, dx = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dopt.dopt_dropout(dopt.DropoutArgs(torch.ones(n, device="cuda"), shown, dropout_of(DROP)), stream=stream())
    leaf = x.clone().requires_grad_()
    (leaf * shown * dy).sum().backward()
    dopt.dopt_dropout(dopt.DropoutArgs(dy, dx, dropout_of(DROP)), stream=stream())
    assert torch.equal(dx, leaf.grad)


def test_dropout_of_a_step_on_the_device():
    """The host's and the device's step add up; a captured dropout follows the device's."""
    n = 4000
    x, y = torch.ones(n, device="cuda"), torch.empty(n, device="cuda")
    at = torch.tensor([4], device="cuda")
    args = dopt.DropoutArgs(x, y, dropout_of(dict(DROP, t=9), d_step=at))
    dopt.dopt_dropout(args, stream=stream())

    def gone(t):
        return O.random16(np.arange(n), 77, 5, t) < O.threshold(0.2)

    assert np.array_equal(y.cpu().numpy() == 0, gone(13))
    args.set_step(0)
    dopt.dopt_dropout(args, stream=stream())
    assert np.array_equal(y.cpu().numpy() == 0, gone(4))
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        dopt.dopt_dropout(args, stream=s)
        at.add_(1)
    for t in (4, 5, 6):
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(y.cpu().numpy() == 0, gone(t))


def test_dropout_far_elements():
    """More than 2^33 elements, in place: the hash's further term, and offsets past 32 bits."""
    n, tail = 2**33 + 5000, 6000
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    dopt.dopt_dropout(dopt.DropoutArgs(x, x, dropout_of(dict(DROP, p=0.5))), stream=stream())
    torch.cuda.synchronize()
    for lo in (0, 2**31 - 3000, 2**32 - 3000, 2**33 - 3000, n - tail):
        got = x[lo:lo + tail].float().cpu().numpy()
        gone = O.random16(np.arange(lo, lo + tail), 77, 5, 13) < 32768
        assert np.array_equal(got == 0, gone) and (got[~gone] == 2).all()


# --------------------------------------------------------------------- norm --

def run_norm(x, dtype, residual=None, drop=None, values=True, codes=True, gain_dtype="f32", pad=0, offset=0, eps=EPS):
    rows, cols = x.shape
    gain = stored(1 + 0.2 * np.random.default_rng(9).standard_normal(cols), gain_dtype)
    stores_h = residual is not None or drop is not None
    a = dict(x=Rows(x, dtype, pad, offset), y=empty(rows, cols, dtype, pad, offset) if values else None,
             h=empty(rows, cols, dtype, pad, offset) if stores_h else None,
             residual=Rows(residual, dtype, pad, offset) if residual is not None else None)
    m = Codes(rows, cols, 1) if codes else None
    rstd = torch.full((rows,), 7.0, device="cuda")
    from matrices_harness import TORCH
    args = dopt.RmsNormArgs(a["x"].view, torch.from_numpy(gain).to(TORCH[gain_dtype]).cuda(), eps,
                            **{k: a[k].view for k in ("y", "h", "residual") if a[k] is not None}, dropout=dropout_of(drop),
                            y8=m.m if m else None, rstd=rstd)
    dopt.dopt_rms_norm(args, stream=stream())
    torch.cuda.synchronize()
    assert all(r is None or r.guards_intact() for r in a.values()) and (m is None or m.guards_intact())
    return gain, a, m, rstd.double().cpu().numpy()


def check_norm(x, dtype, residual=None, drop=None, eps=EPS, **kw):
    gain, a, m, rstd = run_norm(x, dtype, residual, drop, eps=eps, **kw)
    h = x
    if a["h"] is not None:
        want, bound = O.norm_input(x, residual, drop)
        h = a["h"].numpy()
        assert_near(h, want, bound, dtype)
    (r, dr), (y, dy) = O.norm(h, gain, eps)
    assert_near(rstd, r, dr, "f32")
    if a["y"] is not None:
        assert_near(a["y"].numpy(), y, dy, dtype)
    if m is not None:
        check_codes(m.numpy(), m.scale_bytes(), y, dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(rows, cols, dtype):
    x, res = stored(numbers(rows, cols, cols), dtype), stored(numbers(rows, cols, cols + 1), dtype)
    check_norm(x, dtype)
    check_norm(x, dtype, residual=res, codes=False, pad=3, offset=1)
    check_norm(x, dtype, residual=res, drop=DROP, values=False, pad=8)
    check_norm(x, dtype, drop=DROP, gain_dtype=dtype)


def test_norm_many_rows():
    """More rows than CTAs, odd row numbers of an odd length among them."""
    for rows, cols in ((5000, 97), (3000, 513), (2500, 1100)):
        x = stored(numbers(rows, cols, 3), "bf16")
        check_norm(x, "bf16", residual=stored(numbers(rows, cols, 4), "bf16"), drop=DROP)


def test_norm_extremes():
    """Rows of zeros, of squares outside fp32's range, and with infinities and NaN."""
    cols = 700
    x = stored(numbers(8, cols, 1), "f32")
    x[1] = 0
    x[2] *= 1e30
    x[3] = stored(np.full(cols, 2e38), "f32")
    x[4] *= 2.0**-120
    x[5, 3] = np.inf
    x[6, 9] = np.nan
    gain, a, m, rstd = run_norm(x, "f32")
    x, y = a["x"].numpy(), a["y"].numpy()  # x as the array holds it: row 4 has subnormal numbers
    fine = [0, 1, 2, 4, 7]
    (r, dr), (want, dy) = O.norm(x[fine], gain, EPS)
    assert_near(rstd[fine], r, dr, "f32")
    assert_near(y[fine], want, dy, "f32")
    check_codes(m.numpy()[fine], m.scale_bytes()[fine], want, dy)
    # 1 / 2e38 is subnormal: within its last place
    assert abs(rstd[3] * 2e38 - 1) < 1e-6 and np.allclose(y[3], gain, rtol=1e-6)
    assert rstd[5] == 0 and np.isnan(y[5, 3]) and (np.delete(y[5], 3) == 0).all()
    assert np.isnan(rstd[6]) and np.isnan(y[6]).all()
    assert (m.scale_bytes()[6] == 255).all() and m.scale_bytes()[5].tolist() == [255] + [8] * 5


def test_norm_of_far_rows():
    """Rows more than 2^31 bytes apart, in place, forward and backward."""
    rows, cols, ld = 3, 301, 2**30 + 512
    x, dy = stored(numbers(rows, cols, 1), "bf16"), stored(numbers(rows, cols, 2), "bf16")
    whole = torch.zeros(2 * ld + cols + 64, dtype=torch.bfloat16, device="cuda")
    far = whole.as_strided((rows, cols), (ld, 1))
    far.copy_(torch.from_numpy(x))
    m, rstd = Codes(rows, cols), torch.zeros(rows, device="cuda")
    gain = torch.ones(cols, device="cuda")
    dopt.dopt_rms_norm(dopt.RmsNormArgs(far, gain, EPS, y=far, y8=m.m, rstd=rstd), stream=stream())
    (r, dr), (y, d) = O.norm(x, np.ones(cols), EPS)
    assert_near(far.double().cpu().numpy(), y, d, "bf16")
    check_codes(m.numpy(), m.scale_bytes(), y, d)
    assert_near(rstd.double().cpu().numpy(), r, dr, "f32")
    far.copy_(torch.from_numpy(dy))
    h = torch.from_numpy(x).bfloat16().cuda()
    dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(far, h, gain, rstd, far), stream=stream())
    (dh, b), _ = O.norm_backward(dy, x, np.ones(cols), rstd.double().cpu().numpy(), None)
    assert_near(far.double().cpu().numpy(), dh, b, "bf16")
    far.zero_()
    assert not bool(whole.any())


def test_norm_in_place():
    rows, cols = 50, 300
    x, res = stored(numbers(rows, cols, 1), "bf16"), stored(numbers(rows, cols, 2), "bf16")
    gain, a, _, _ = run_norm(x, "bf16", res, DROP, codes=False)
    xs, rs = Rows(x, "bf16"), Rows(res, "bf16")
    dopt.dopt_rms_norm(dopt.RmsNormArgs(xs.view, torch.from_numpy(gain).float().cuda(), EPS, residual=rs.view, h=rs.view, y=xs.view,
                                        dropout=dropout_of(DROP)), stream=stream())
    assert np.array_equal(rs.numpy(), a["h"].numpy()) and np.array_equal(xs.numpy(), a["y"].numpy())


def test_norm_together_is_norm_apart():
    """Dropout and the residual's addition, then the norm of what they left: the same bits as in one call."""
    x, res = stored(numbers(60, 1000, 1), "bf16"), stored(numbers(60, 1000, 2), "bf16")
    _, a, m, rstd = run_norm(x, "bf16", res, DROP)
    h = empty(60, 1000, "bf16")
    dopt.dopt_dropout(dopt.DropoutArgs(Rows(x, "bf16").view.contiguous(), h.view, dropout_of(DROP),
                                       residual=Rows(res, "bf16").view.contiguous()), stream=stream())
    assert np.array_equal(h.numpy(), a["h"].numpy())
    _, b, n, rstd2 = run_norm(h.numpy(), "bf16")
    assert np.array_equal(a["y"].numpy(), b["y"].numpy()) and np.array_equal(m.numpy(), n.numpy()) and np.array_equal(rstd, rstd2)


# ----------------------------------------------------------- backward pass --

def run_backward(h, dy, dtype, dres=None, drop=None, add=False, gain_dtype="f32", pad=0, offset=0, in_place=False, dgain=True):
    rows, cols = h.shape
    rng = np.random.default_rng(4)
    gain = stored(1 + 0.2 * rng.standard_normal(cols), gain_dtype)
    old = stored(rng.standard_normal(cols), "f32")
    rstd = stored(O.norm(h, gain, EPS)[0][0], "f32")
    a = dict(h=Rows(h, dtype, pad, offset), dy=Rows(dy, dtype, pad, offset),
             dres=Rows(dres, dtype, pad, offset) if dres is not None else None)
    a["dh"] = (a["dres"] or a["dy"]) if in_place else empty(rows, cols, dtype, pad, offset)
    a["dx"] = None if drop is None else a["dy"] if in_place and dres is not None else empty(rows, cols, dtype, pad, offset)
    from matrices_harness import TORCH
    out = Rows(old[None], "f32")
    size = dopt.dopt_rms_norm_workspace_bytes(rows, cols)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    args = dopt.RmsNormBackwardArgs(a["dy"].view, a["h"].view, torch.from_numpy(gain).to(TORCH[gain_dtype]).cuda(),
                                    torch.from_numpy(rstd).float().cuda(), a["dh"].view,
                                    dres=None if dres is None else a["dres"].view, dropout=dropout_of(drop),
                                    dx=None if drop is None else a["dx"].view, dgain=out.view[0] if dgain else None, accumulate=add,
                                    workspace=ws, workspace_bytes=size)
    dopt.dopt_rms_norm_backward(args, stream=stream())
    torch.cuda.synchronize()
    assert all(r is None or r.guards_intact() for r in a.values()) and out.guards_intact() and bool((ws[size:] == 0xFF).all())
    (dh, b), (dg, bg) = O.norm_backward(dy, h, gain, rstd, dres)
    assert_near(a["dh"].numpy(), dh, b, dtype)
    if drop is not None:
        dx, bx = O.dropout(dh, drop)
        scale = 65536 / (65536 - O.threshold(drop["p"]))
        assert_near(a["dx"].numpy(), dx, bx + b * scale, dtype)
    got = out.numpy()[0]
    if dgain:
        assert_near(got, dg + old if add else dg, bg + (O.U * np.abs(dg + old) if add else 0), "f32")
    else:
        assert np.array_equal(got, old)
    return a, got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_backward(rows, cols, dtype):
    h, dy, dres = (stored(numbers(rows, cols, cols + k), dtype) for k in range(3))
    run_backward(h, dy, dtype)
    run_backward(h, dy, dtype, dres=dres, add=True, pad=3, offset=1, gain_dtype=dtype)
    run_backward(h, dy, dtype, dres=dres, drop=DROP, pad=8)
    run_backward(h, dy, dtype, dres=dres, drop=DROP, in_place=True, dgain=False)
    run_backward(h, dy, dtype, drop=DROP, in_place=True)


@pytest.mark.parametrize("rows,cols", [(5000, 97), (3000, 513), (2500, 1100), (1300, 2050)])
def test_norm_backward_many_rows(rows, cols):
    h, dy, dres = (stored(numbers(rows, cols, k), "bf16") for k in range(3))
    _, first = run_backward(h, dy, "bf16", dres=dres, drop=DROP)
    _, again = run_backward(h, dy, "bf16", dres=dres, drop=DROP)
    assert np.array_equal(first, again)


def test_norm_backward_with_a_dropout_of_nothing():
    """p = 0 in both passes: dx is dh."""
    h, dy = stored(numbers(70, 300, 1), "bf16"), stored(numbers(70, 300, 2), "bf16")
    a, _ = run_backward(h, dy, "bf16", drop=dict(DROP, p=0.0))
    assert np.array_equal(a["dx"].numpy(), a["dh"].numpy())


def test_norm_backward_of_no_rows():
    gain, dgain = torch.ones(9, device="cuda"), torch.full((9,), 3.0, device="cuda")
    none, r = torch.zeros(0, 9, device="cuda"), torch.zeros(0, device="cuda")
    for add, want in ((True, 3.0), (False, 0.0)):
        dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(none, none, gain, r, none, dgain=dgain, accumulate=add), stream=stream())
        assert bool((dgain == want).all())


def test_norm_backward_is_torchs():
    """Against torch's own gradients of the formula, in fp64."""
    rows, cols = 30, 500
    h, dy = stored(numbers(rows, cols, 1, 0.5), "f32"), stored(numbers(rows, cols, 2, 0.5), "f32")
    a, dgain = run_backward(h, dy, "f32")
    gain = stored(1 + 0.2 * np.random.default_rng(4).standard_normal(cols), "f32")
    x, g = torch.from_numpy(h).requires_grad_(), torch.from_numpy(gain).requires_grad_()
    (x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * g * torch.from_numpy(dy)).sum().backward()
    scale = np.abs(x.grad.numpy()).max(1, keepdims=True)
    assert np.abs((a["dh"].numpy() - x.grad.numpy()) / scale).max() < 2e-5
    assert np.abs(dgain - g.grad.numpy()).max() < 2e-5 * np.abs(g.grad.numpy()).max()
