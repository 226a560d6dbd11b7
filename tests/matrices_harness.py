"""Arrays inside guards of a known pattern, 8-bit matrices, and reads back,
for the GPU tests of the 8-bit matrices, the norm and dropout."""

import numpy as np
import torch

from oracle import matrices as O

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GUARD = 64


class Rows:
    """rows x cols values, `pad` elements between rows, `offset` elements past an aligned start, inside guards."""

    def __init__(self, values, dtype, pad=0, offset=0):
        values = torch.as_tensor(np.asarray(values)) if not torch.is_tensor(values) else values
        rows, cols = values.shape
        self.whole = torch.full((GUARD + offset + rows * (cols + pad) + GUARD,), 77, dtype=TORCH.get(dtype, dtype), device="cuda")
        self.view = self.whole[GUARD + offset:][: rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.view.copy_(values)
        self.inside = torch.zeros_like(self.whole, dtype=torch.bool)
        self.inside[GUARD + offset:][: rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True

    def guards_intact(self):
        return bool((self.whole[~self.inside] == 77).all())

    def numpy(self):
        torch.cuda.synchronize()
        return self.view.double().cpu().numpy()


def empty(rows, cols, dtype, pad=0, offset=0):
    return Rows(torch.full((rows, cols), 55.0), dtype, pad, offset)


class Codes:
    """A rows x cols 8-bit matrix (codes on 16-byte boundaries, `pad` * 16 more bytes per row), filled with a pattern."""

    def __init__(self, rows, cols, pad=0):
        import mixed_precision_adam_gb300 as dopt
        ld = -(-cols // 16) * 16 + 16 * pad
        self.rows, self.cols = rows, cols
        self.whole = torch.full((GUARD + rows * ld + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
        self.codes = self.whole[GUARD:][: rows * ld].view(rows, ld)[:, :cols]
        self.inside = torch.zeros_like(self.whole, dtype=torch.bool)
        self.inside[GUARD:][: rows * ld].view(rows, ld)[:, :cols] = True
        self.scales = torch.full((dopt.dopt_matrix8_scale_bytes(rows, cols),), 0x5A, dtype=torch.uint8, device="cuda")
        self.places = O.scale_places(rows, cols)
        self.m = dopt.Matrix8(self.codes, self.scales)

    def fill(self, values, square=False):
        """The nearest codes of `values`; returns what they stand for."""
        s = O.scales(values, square)
        q = O.rounded(values, s)
        unit = 2.0 ** (O.per_column(s, self.cols) - 127.0)
        self.codes.copy_(torch.from_numpy(q / unit).to(torch.float8_e4m3fn).view(torch.uint8))
        self.set_scales(s)
        return q

    def set_scales(self, s):
        host = self.scales.cpu().numpy()
        host[self.places] = s
        self.scales.copy_(torch.from_numpy(host))

    def scale_bytes(self):
        torch.cuda.synchronize()
        return self.scales.cpu().numpy()[self.places]

    def numpy(self):
        return O.values(self.codes.cpu().numpy(), self.scale_bytes())

    def guards_intact(self):
        """Neither the bytes around the codes nor the scale bytes of rows and blocks that are not there are written."""
        s = self.scales.cpu().numpy().copy()
        s[self.places] = 0x5A
        return bool((self.whole[~self.inside] == 0x5A).all()) and bool((s == 0x5A).all())


def numbers(rows, cols, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, cols)))
    return x * np.exp(rng.standard_normal((rows, 1)))


def stored(x, dtype):
    """x as values of a type, in float64."""
    return torch.from_numpy(np.asarray(x)).to(TORCH[dtype]).double().numpy()


def check_codes(got_values, got_scale, want, bound):
    """Codes and scales are those of some values within `bound` of `want`: the roundings are monotone."""
    low, high = np.maximum(np.abs(want) - bound, 0), np.abs(want) + bound
    assert ((got_scale >= O.scales(low)) & (got_scale <= O.scales(high))).all()
    lo, hi = O.rounded(want - bound, got_scale), O.rounded(want + bound, got_scale)
    ok = ((got_values >= lo) & (got_values <= hi)) | (np.isnan(got_values) & np.isnan(lo))
    assert ok.all(), (np.argwhere(~ok)[:4], got_values[~ok][:4], lo[~ok][:4], hi[~ok][:4])
