"""Seeded lists of tensors on the GPU for the tests of the step over a list:
every array sits between guard elements, at a chosen offset from an aligned
address, and what a call left is compared with the 64-bit restatement."""

import numpy as np
import torch

from oracle import tensors as O

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "u8": torch.uint8}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
GUARD = 64


class Array:
    """n elements at `offset` elements past an aligned start, inside guards of a known pattern."""

    def __init__(self, values, dtype, offset=0):
        n = values.numel()
        self.whole = torch.full((GUARD + offset + n + GUARD,), 77, dtype=dtype, device="cuda")
        self.lo, self.hi = GUARD + offset, GUARD + offset + n
        self.view = self.whole[self.lo:self.hi]
        self.view.copy_(values)

    def guards_intact(self):
        return bool((self.whole[: self.lo] == 77).all()) and bool((self.whole[self.hi:] == 77).all())

    def numpy(self):
        return (self.view.float() if self.view.dtype != torch.uint8 else self.view).cpu().numpy()


class Case:
    """tensors: dicts of numel, param, grad ("f32", "bf16", "f16"), moments (32 or 8), offset (of every array, in
    elements) and offsets (of the arrays named, instead), wd_mult, zero (share of zero grads and moments)."""

    def __init__(self, tensors, seed, grad_size=1e-2, scale=1.0):
        import mixed_precision_adam_gb300 as dopt
        gen = torch.Generator().manual_seed(seed)
        self.spec, self.arrays, entries = tensors, [], []
        for t in tensors:
            n, offs = t["numel"], t.get("offsets", {})

            def off(name, default=t.get("offset", 0), offs=offs):
                return offs.get(name, default)

            size = torch.exp(torch.randn(n, generator=gen)) * grad_size
            size *= torch.rand(n, generator=gen) >= t.get("zero", 0.0)
            a = dict(grad=Array(torch.randn(n, generator=gen) * size * scale, TORCH[t["grad"]], off("grad")))
            w = torch.randn(n, generator=gen) * 0.05
            a["param"] = Array(w.to(TORCH[t["param"]]), TORCH[t["param"]], off("param"))
            if t["param"] != "f32":
                a["master"] = Array(w, torch.float32, off("master"))
            m, v = torch.randn(n, generator=gen) * size * 0.3, torch.rand(n, generator=gen) * size * size
            if t["moments"] == 32:
                a["exp_avg"] = Array(m, torch.float32, off("exp_avg"))
                a["exp_avg_sq"] = Array(v, torch.float32, off("exp_avg_sq"))
            else:
                ms, vs = O.m_scale(m.double().numpy()), O.v_scale(v.double().numpy())
                a["exp_avg_scale"] = Array(torch.from_numpy(ms), torch.uint8, off("exp_avg_scale"))
                a["exp_avg_sq_scale"] = Array(torch.from_numpy(vs), torch.uint8, off("exp_avg_sq_scale"))
                mc = torch.randint(0, 255, (n,), generator=gen)
                mc = torch.where(mc == 127, 3, mc)  # e4m3's NaN codes are never stored
                vc = torch.randint(0, 256, (n,), generator=gen)
                zero = size == 0
                a["exp_avg"] = Array(torch.where(zero, 0, mc), torch.uint8, off("exp_avg"))
                a["exp_avg_sq"] = Array(torch.where(zero, 0, vc), torch.uint8, off("exp_avg_sq"))
            self.arrays.append(a)
            entries.append(dict({k: x.view for k, x in a.items()}, wd_mult=t.get("wd_mult", 1.0)))
        self.list = dopt.TensorList(entries)
        self.before = self.values()

    def values(self):
        """Every array as numpy: codes as they are, floats as float32."""
        torch.cuda.synchronize()
        return [{k: x.numpy().copy() for k, x in a.items()} for a in self.arrays]

    def moments(self, vals, k):
        if self.spec[k]["moments"] == 32:
            return vals["exp_avg"].astype(np.float64), vals["exp_avg_sq"].astype(np.float64)
        return (O.m_values(vals["exp_avg"], vals["exp_avg_scale"]),
                O.v_values(vals["exp_avg_sq"], vals["exp_avg_sq_scale"]))

    def weights(self, vals):
        return vals["master"] if "master" in vals else vals["param"]

    def check_guards(self):
        for k, a in enumerate(self.arrays):
            for name, x in a.items():
                assert x.guards_intact(), (k, name)

    def check_unchanged(self, names=None):
        for k, (a, b) in enumerate(zip(self.before, self.values())):
            for name in names or a:
                assert np.array_equal(a[name].view(np.uint8), b[name].view(np.uint8)), (k, name)
        self.check_guards()

    def check_step(self, step, inv_scale=1.0, coef=1.0, seed=0, hp=HP):
        """What one step left against the 64-bit step from what was there before; the new values become
        the next step's start."""
        after = self.values()
        for k, (a, b) in enumerate(zip(self.before, after)):
            t = self.spec[k]
            m, v = self.moments(a, k)
            w = self.weights(a)
            (w1, m1, v1), (dw, dm, dv) = O.adamw(w, a["grad"], m, v, hp, step, inv_scale, coef, t.get("wd_mult", 1.0))
            got = self.weights(b).astype(np.float64)
            ok = np.abs(got - w1) <= dw
            assert ok.all(), (k, "weight", np.flatnonzero(~ok)[:5], got[~ok][:3], w1[~ok][:3])
            if "master" in b:
                cast = torch.from_numpy(b["master"]).to(TORCH[t["param"]]).float().numpy()
                assert np.array_equal(cast, b["param"]), (k, "param")
            assert np.array_equal(a["grad"], b["grad"]), (k, "grad")
            if t["moments"] == 32:
                for name, x, d in (("exp_avg", m1, dm), ("exp_avg_sq", v1, dv)):
                    ok = np.abs(b[name] - x) <= d
                    assert ok.all(), (k, name, np.flatnonzero(~ok)[:5])
            else:
                check_codes(b, m1, dm, v1, dv, O.rounding_fraction(t["numel"], k, step, seed), k)
        self.check_guards()
        self.before = after


def check_codes(b, m1, dm, v1, dv, fraction, k=0):
    """Codes and scales are those of some moments within dm, dv of m1, v1: the roundings are monotone, so each
    stored value lies between those of the two ends."""
    for name, scale, lo, hi in (("exp_avg_scale", O.m_scale, np.maximum(np.abs(m1) - dm, 0), np.abs(m1) + dm),
                                ("exp_avg_sq_scale", O.v_scale, np.maximum(v1 - dv, 0), v1 + dv)):
        s = b[name]
        assert len(s) == -(-len(m1) // O.BLOCK)
        assert ((s >= scale(lo)) & (s <= scale(hi))).all(), (k, name, s[:8], scale(lo)[:8], scale(hi)[:8])
    got = O.m_values(b["exp_avg"], b["exp_avg_scale"])
    lo, hi = O.m_rounded(m1 - dm, b["exp_avg_scale"]), O.m_rounded(m1 + dm, b["exp_avg_scale"])
    ok = (got >= lo) & (got <= hi)
    assert ok.all(), (k, "exp_avg", np.flatnonzero(~ok)[:5], got[~ok][:3], lo[~ok][:3], hi[~ok][:3])
    got = O.v_values(b["exp_avg_sq"], b["exp_avg_sq_scale"])
    lo = O.v_rounded(np.maximum(v1 - dv, 0), b["exp_avg_sq_scale"], fraction)
    hi = O.v_rounded(v1 + dv, b["exp_avg_sq_scale"], fraction)
    hi = np.where(v1 == 0, 0.0, hi)
    lo = np.where(v1 == 0, 0.0, lo)
    ok = (got >= lo) & (got <= hi)
    assert ok.all(), (k, "exp_avg_sq", np.flatnonzero(~ok)[:5], got[~ok][:3], lo[~ok][:3], hi[~ok][:3])
