"""Arguments of the 8-bit operators that are of another kind than asked for
are refused as the others are, with a DoptError that names them."""

import torch

from test_matrix8_host import dopt, refused, u8


def test_what_is_no_tensor_or_no_handle():
    x, g, m = torch.zeros(5, 40), torch.ones(40), dopt.Matrix8(u8(5, 48)[:, :40], u8(512))
    drop, r = dopt.Dropout(0.1, 1), torch.zeros(5)
    for name, call in (
            ("x is", lambda: dopt.DropoutArgs([1.0], x, drop)),
            ("x is", lambda: dopt.DropoutArgs(None, x, drop)),
            ("x is", lambda: dopt.DropoutArgs(x.numpy(), x, drop)),
            ("x is", lambda: dopt.DropoutArgs(x.int(), x, drop)),
            ("x is", lambda: dopt.DropoutArgs(x.t(), x, drop)),
            ("residual is", lambda: dopt.DropoutArgs(x, x, drop, residual=3)),
            ("dropout is", lambda: dopt.DropoutArgs(x, x, 0.1)),
            ("x is", lambda: dopt.RmsNormArgs(5, g, 1e-6, y=x)),
            ("gain is", lambda: dopt.RmsNormArgs(x, 1.0, 1e-6, y=x)),
            ("y8 is", lambda: dopt.RmsNormArgs(x, g, 1e-6, y8=u8(5, 48))),
            ("dropout is", lambda: dopt.RmsNormArgs(x, g, 1e-6, y=x, h=x.clone(), dropout=0.1)),
            ("dropout is", lambda: dopt.RmsNormBackwardArgs(x, x, g, r, x, dropout=dict(p=0.1))),
            ("h is", lambda: dopt.RmsNormBackwardArgs(x, None, g, r, x)),
            ("rstd is", lambda: dopt.RmsNormBackwardArgs(x, x, g, None, x)),
            ("matrix 0: out is", lambda: dopt.MatrixList([dict(values=x, out=u8(5, 48))])),
            ("matrix 0: out_t is", lambda: dopt.MatrixList([dict(values=x, out_t=(u8(40, 16), u8(512)))])),
            ("a is", lambda: dopt.dopt_matrix8_multiply(x, m, torch.zeros(5, 5))),
            ("b is", lambda: dopt.dopt_matrix8_multiply(m, None, torch.zeros(5, 5))),
            ("d is", lambda: dopt.dopt_matrix8_multiply(m, m, None))):
        assert name in refused(dopt.E_INVALID, call)
