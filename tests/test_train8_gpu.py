"""The 8-bit operators as a training step uses them, one after another:
dropout, the residual and the norm to codes, a product with packed weights,
the backward pass's two products and the norm's, the gains' and weights'
grads into a list's step, and the weights packed again.  Each against the
64-bit restatement on what the one before left, eager and captured."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from matrices_harness import check_codes  # noqa: E402
from oracle import matrices as O  # noqa: E402

HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
T, D, F = 200, 260, 390  # tokens, width, outputs; none a multiple of 128
EPS = 1e-6


def codes(rows, cols):
    m = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda")[:, :cols]
    return dopt.Matrix8(m, torch.zeros(dopt.dopt_matrix8_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda"))


def scale_bytes(m):
    return m.scales.cpu().numpy()[O.scale_places(m.rows, m.cols)]


def values(m):
    return O.values(m.codes.cpu().numpy(), scale_bytes(m))


def host(t):
    return t.double().cpu().numpy()


class Step:
    """y = norm(dropout(x) + residual) W^T; x's, the residual's, the gain's and W's gradients; the step."""

    def __init__(self, seed):
        gen = torch.Generator("cuda").manual_seed(seed)

        def normal(*s):
            return torch.randn(*s, generator=gen, device="cuda")

        self.x, self.res = normal(T, D).bfloat16(), normal(T, D).bfloat16()
        self.dy, self.dres = (normal(T, F) * 1e-2).bfloat16(), (normal(T, D) * 1e-2).bfloat16()
        self.w32, self.gain = normal(F, D) * 0.05, 1 + 0.1 * normal(D)
        self.w = self.w32.bfloat16()
        self.applied = torch.zeros(1, dtype=torch.int64, device="cuda")
        e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.h, self.n, self.y, self.dn, self.dh, self.dx = e(T, D), e(T, D), e(T, F), e(T, D), e(T, D), e(T, D)
        self.rstd, self.dw, self.dgain = e(T, t=torch.float32), e(F, D, t=torch.float32), e(D, t=torch.float32)
        self.n8, self.n8t, self.dy8, self.dy8t = codes(T, D), codes(D, T), codes(T, F), codes(F, T)
        self.w8, self.w8t = codes(F, D), codes(D, F)
        drop = dopt.Dropout(0.1, 99, site=2, d_step=self.applied)
        self.forward = dopt.RmsNormArgs(self.x, self.gain, EPS, residual=self.res, dropout=drop, h=self.h, y=self.n, y8=self.n8,
                                        rstd=self.rstd)
        size = dopt.dopt_rms_norm_workspace_bytes(T, D)
        self.backward = dopt.RmsNormBackwardArgs(self.dn, self.h, self.gain, self.rstd, self.dh, dres=self.dres, dropout=drop, dx=self.dx,
                                                 dgain=self.dgain, workspace=e(size, t=torch.uint8), workspace_bytes=size)
        self.pack_w = dopt.MatrixList([dict(values=self.w32, block=dopt.BLOCK_SQUARE, out=self.w8, out_t=self.w8t)])
        self.pack_grads = dopt.MatrixList([dict(values=self.n, out_t=self.n8t), dict(values=self.dy, out=self.dy8, out_t=self.dy8t)])
        state = [dict(param=self.w, grad=self.dw, master=self.w32, exp_avg=torch.zeros(F, D, device="cuda"),
                      exp_avg_sq=torch.zeros(F, D, device="cuda")),
                 dict(param=self.gain, grad=self.dgain, exp_avg=torch.zeros(D, device="cuda"), exp_avg_sq=torch.zeros(D, device="cuda"),
                      wd_mult=0.0)]
        self.list = dopt.TensorList(state)
        self.ws = e(dopt.dopt_tensors_workspace_bytes(2), t=torch.uint8)
        self.grad_norm = e(1, t=torch.float32)

    def run(self, s):
        dopt.dopt_matrix8_pack(self.pack_w, stream=s)
        dopt.dopt_rms_norm(self.forward, stream=s)
        dopt.dopt_matrix8_multiply(self.n8, self.w8, self.y, stream=s)
        dopt.dopt_matrix8_pack(self.pack_grads, stream=s)
        dopt.dopt_matrix8_multiply(self.dy8, self.w8t, self.dn, stream=s)
        dopt.dopt_matrix8_multiply(self.dy8t, self.n8t, self.dw, stream=s)
        dopt.dopt_rms_norm_backward(self.backward, stream=s)
        dopt.dopt_tensors_step(self.list, HP, 1, self.ws, self.ws.numel(), max_norm=1.0, d_step=self.applied, d_norm=self.grad_norm,
                               stream=s)

    def check(self, w_before, gain_before, t):
        drop = dict(p=0.1, seed=99, site=2, t=t)
        w, gain = host(w_before), host(gain_before)
        for m, v in ((self.w8, w), (self.w8t, w.T)):
            assert np.array_equal(values(m), O.rounded(v, O.scales(v, True)))
        want, bound = O.norm_input(host(self.x), host(self.res), drop)
        h = host(self.h)
        assert O.near(h, want, bound, "bf16").all()
        (r, dr), (n, dn) = O.norm(h, gain, EPS)
        assert O.near(host(self.rstd), r, dr, "f32").all() and O.near(host(self.n), n, dn, "bf16").all()
        check_codes(values(self.n8), scale_bytes(self.n8), n, dn)
        for m, v in ((self.n8t, host(self.n).T), (self.dy8, host(self.dy)), (self.dy8t, host(self.dy).T)):
            assert np.array_equal(values(m), O.rounded(v, O.scales(v)))
        for got, a, b, dtype in ((self.y, self.n8, self.w8, "bf16"), (self.dn, self.dy8, self.w8t, "bf16"), (self.dw, self.dy8t, self.n8t, "f32")):
            want, bound = O.product(values(a), values(b))
            assert O.near(host(got), want, bound, dtype).all()
        (dh, b), (dg, bg) = O.norm_backward(host(self.dn), h, gain, host(self.rstd), host(self.dres))
        assert O.near(host(self.dh), dh, b, "bf16").all() and O.near(host(self.dgain), dg, bg, "f32").all()
        dx, bx = O.dropout(dh, drop)
        assert O.near(host(self.dx), dx, bx + b * 1.2, "bf16").all()
        norm = np.sqrt((host(self.dw) ** 2).sum() + (host(self.dgain) ** 2).sum())
        assert abs(float(self.grad_norm) / norm - 1) < 1e-5
        assert not torch.equal(self.w32, w_before) and torch.isfinite(self.w32).all()
        # the 8-bit gradients are near the exact ones: every factor rounded by at most 2^-4 of itself, or 2^-10 of its
        # block's largest value, which for normal numbers adds to less than a tenth of the whole
        exact = host(self.dy).T @ n
        assert np.linalg.norm(host(self.dw) - exact) < 0.1 * np.linalg.norm(exact)


def test_a_training_step():
    st = Step(1)
    for t in range(3):
        w, gain = st.w32.clone(), st.gain.clone()
        st.run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert int(st.applied) == t + 1
        st.check(w, gain, t)


def test_captured_steps():
    """Two models' steps as graphs, replayed in turn with new inputs and at once; the same bits as eager steps."""
    pairs = []
    for seed in (1, 2):
        eager, cap = Step(seed), Step(seed)
        s = torch.cuda.Stream()
        eager.run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cap.run(s)
        g.replay()
        pairs.append((eager, cap, g))
    for k in range(3):
        new = torch.randn(T, D, device="cuda").bfloat16()
        torch.cuda.synchronize()
        for eager, cap, g in pairs:
            eager.x.copy_(new)
            cap.x.copy_(new)
            torch.cuda.synchronize()
            g.replay()
            eager.run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        for eager, cap, _ in pairs:
            assert int(eager.applied) == int(cap.applied) == k + 2
            for name in ("y", "dx", "dh", "dw", "dgain", "w32", "gain", "w"):
                assert torch.equal(getattr(eager, name), getattr(cap, name)), (k, name)
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, _, g), s in zip(pairs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for eager, _, _ in pairs:
            eager.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for eager, cap, _ in pairs:
        assert torch.equal(eager.w32, cap.w32) and torch.equal(eager.dx, cap.dx)
