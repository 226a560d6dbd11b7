"""The 8-bit matrices, their products, the norm and dropout without a GPU: the
struct layouts, the refusals of every entry point (before any device work),
and the 64-bit restatement, itself checked against brute force and
differences."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import matrices as O

dopt = pytest.importorskip("mixed_precision_adam_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ["dopt_matrix8", "dopt_matrix_values", "dopt_drop", "dopt_dropout_args", "dopt_rows", "dopt_rms_norm_args",
           "dopt_rms_norm_backward_args"]


def refused(status, call):
    with pytest.raises(dopt.DoptError) as err:
        call()
    assert err.value.status == status, err.value
    return str(err.value)


@pytest.mark.parametrize("name", STRUCTS)
def test_binding_structs_match_header(tmp_path, name):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    cls = getattr(dopt, name)
    body = "".join(f'printf("{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_)
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dopt.h"\nint main(void) {'
                                  f'printf("size %zu\\n", sizeof({name}));{body}return 0;}}')
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    for line in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split("\n"):
        if line:
            field, value = line.split()
            assert (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset) == int(value), line


def test_constants_match_header():
    text = open(os.path.join(ROOT, "include", "dopt.h")).read()
    assert f"#define DOPT_MATRIX_BLOCK {dopt.MATRIX_BLOCK}\n" in text
    assert f"#define DOPT_NORM_MAX_COLS {dopt.NORM_MAX_COLS}\n" in text


def test_sizes():
    assert [dopt.dopt_matrix8_scale_bytes(*s) for s in ((0, 5), (1, 1), (128, 512), (129, 512), (128, 513), (300, 2048))] \
        == [0, 512, 512, 1024, 1024, 3 * 4 * 512]
    for rows, cols in ((1, 1), (130, 700), (31, 2049)):
        assert dopt.dopt_matrix8_scale_bytes(rows, cols) == O.scale_size(rows, cols) > O.scale_places(rows, cols).max()
    refused(dopt.E_INVALID, lambda: dopt.dopt_matrix8_scale_bytes(-1, 3))
    refused(dopt.E_SIZE, lambda: dopt.dopt_matrix8_scale_bytes(1, 2**31))
    assert dopt.dopt_rms_norm_workspace_bytes(0, 5) >= 16
    assert dopt.dopt_rms_norm_workspace_bytes(10**9, 16384) < 2**26
    for bad in ((-1, 5), (5, 16385), (2**31, 5)):
        with pytest.raises(dopt.DoptError):
            dopt.dopt_rms_norm_workspace_bytes(*bad)


def matrix(rows=40, cols=300, ld=304, codes=4096, scales=8192):
    return dopt.dopt_matrix8(rows, cols, ld, codes, scales)


BAD_MATRICES = [(dict(codes=None), "E_INVALID"), (dict(scales=None), "E_INVALID"), (dict(codes=4104), "E_ALIGN"),
                (dict(scales=8200), "E_ALIGN"), (dict(ld=288), "E_INVALID"), (dict(ld=301), "E_ALIGN")]


def multiply(a, b, d=1 << 20, dtype=0, ldd=64, accumulate=0):
    return lambda: dopt._check(dopt._c["dopt_matrix8_multiply"](ctypes.byref(a), ctypes.byref(b), d, dtype, ldd,
                                                               accumulate, None))


def test_refused_products():
    a, b = matrix(), matrix(rows=50)
    for change, status in BAD_MATRICES:
        refused(getattr(dopt, status), multiply(matrix(**change), b))
        refused(getattr(dopt, status), multiply(a, matrix(rows=50, **change)))
    refused(dopt.E_INVALID, multiply(a, matrix(cols=301)))
    refused(dopt.E_INVALID, multiply(matrix(rows=-1), b))
    refused(dopt.E_SIZE, multiply(matrix(rows=2**31), b))
    refused(dopt.E_INVALID, multiply(a, b, d=None))
    refused(dopt.E_INVALID, multiply(a, b, dtype=3))
    refused(dopt.E_INVALID, multiply(a, b, ldd=49))
    refused(dopt.E_SIZE, multiply(a, b, ldd=2**41))
    big = dict(rows=2**31 - 1, cols=2**31 - 1, ld=2**31)
    refused(dopt.E_SIZE, multiply(matrix(**big), matrix(**dict(big, rows=1))))
    refused(dopt.E_ALIGN, multiply(a, b, d=(1 << 20) + 2))
    refused(dopt.E_ALIGN, multiply(a, b, d=(1 << 20) + 1, dtype=1))
    fn = dopt._c["dopt_matrix8_multiply"]
    refused(dopt.E_INVALID, lambda: dopt._check(fn(None, ctypes.byref(b), 1 << 20, 0, 64, 0, None)))
    refused(dopt.E_INVALID, lambda: dopt._check(fn(ctypes.byref(a), None, 1 << 20, 0, 64, 0, None)))
    # nothing to do: no pointer is looked at
    for m in (matrix(rows=0, codes=None), matrix(rows=0, ld=0)):
        multiply(m, b)()
        multiply(b, m)()


def values(rows=40, cols=300, ld=300, dtype=0, block=0, at=1 << 20, out=None, out_t=None):
    none = dopt.dopt_matrix8()
    return dopt.dopt_matrix_values(rows, cols, ld, dtype, block, at, out or none, out_t or none)


def test_refused_packs():
    def call(m, fns=("dopt_matrix8_pack", "dopt_matrix8_unpack"), status=dopt.E_INVALID):
        for fn in fns:
            text = refused(status, lambda: dopt._check(dopt._c[fn]((dopt.dopt_matrix_values * 2)(good, m), 2, None)))
            assert "matrix 1" in text

    good = values(rows=0, out=matrix())
    for change, status in BAD_MATRICES[1:]:
        call(values(out=matrix(**change)), status=getattr(dopt, status))
        call(values(out_t=matrix(**dict(dict(rows=300, cols=40, ld=48), **{k: v if k != "ld" else 32 if v < 300 else 41
                                                                          for k, v in change.items()}))),
             ("dopt_matrix8_pack",), getattr(dopt, status))
    for bad in (values(), values(out=matrix(rows=41)), values(out=matrix(cols=299)), values(rows=-1, out=matrix()),
                values(dtype=5, out=matrix()), values(block=2, out=matrix()), values(ld=299, out=matrix()),
                values(at=None, out=matrix())):
        call(bad)
    call(values(out=matrix(), out_t=matrix()), ("dopt_matrix8_pack",))
    call(values(dtype=2, out=matrix()), ("dopt_matrix8_unpack",))      # fp16 is not exact
    call(values(out_t=matrix(300, 40, 48)), ("dopt_matrix8_unpack",))  # there is nothing to unpack
    call(values(at=(1 << 20) + 2, out=matrix()), status=dopt.E_ALIGN)
    call(values(rows=2**31, out=matrix()), status=dopt.E_SIZE)
    call(values(ld=2**41, out=matrix()), status=dopt.E_SIZE)
    big = matrix(rows=2**31 - 1, cols=2**31 - 1, ld=2**31)
    call(values(rows=2**31 - 1, cols=2**31 - 1, ld=2**31, out=big), status=dopt.E_SIZE)
    for fn in ("dopt_matrix8_pack", "dopt_matrix8_unpack"):
        refused(dopt.E_INVALID, lambda: dopt._check(dopt._c[fn](None, 1, None)))
        refused(dopt.E_INVALID, lambda: dopt._check(dopt._c[fn](None, -1, None)))
        assert dopt._c[fn](None, 0, None) == 0


def drop_args(**kw):
    drop = dopt.dopt_drop(kw.pop("p", 0.1), 1, 2, 3, kw.pop("d_step", None))
    e = dict(numel=100, dtype=1, x=4096, residual=None, y=8192)
    e.update(kw)
    return dopt.dopt_dropout_args(e["numel"], e["dtype"], 0, e["x"], e["residual"], e["y"], drop)


BAD_DROPS = [(dict(p=-0.1), "E_INVALID"), (dict(p=1.0), "E_INVALID"), (dict(p=float("nan")), "E_INVALID"),
             (dict(p=1 - 2.0**-18), "E_INVALID"), (dict(d_step=12), "E_ALIGN")]


@pytest.mark.parametrize("change,status", BAD_DROPS + [
    (dict(numel=-1), "E_INVALID"), (dict(dtype=3), "E_INVALID"), (dict(x=None), "E_INVALID"), (dict(y=None), "E_INVALID"),
    (dict(x=4097), "E_ALIGN"), (dict(y=8193), "E_ALIGN"), (dict(residual=7), "E_ALIGN"), (dict(numel=2**60), "E_SIZE")])
def test_refused_dropout(change, status):
    a = drop_args(**change)
    refused(getattr(dopt, status), lambda: dopt._check(dopt._c["dopt_dropout"](ctypes.byref(a), None)))
    assert dopt._c["dopt_dropout"](ctypes.byref(drop_args(numel=0, x=None, y=None)), None) == 0
    refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_dropout"](None, None)))


def norm_args(**kw):
    e = dict(rows=4, cols=300, dtype=1, gain_dtype=0, x=4096, residual=None, h=None, y=8192, gain=16384, y8=None, rstd=None,
             eps=1e-6, p=0.0, d_step=None, ld=300)
    e.update(kw)
    r = [dopt.dopt_rows(e[k], e["ld"]) for k in ("x", "residual", "h", "y")]
    a = dopt.dopt_rms_norm_args(e["rows"], e["cols"], e["dtype"], e["gain_dtype"], *r, e["gain"],
                                ctypes.pointer(e["y8"]) if e["y8"] else None, e["rstd"], e["eps"],
                                dopt.dopt_drop(e["p"], 1, 2, 3, e["d_step"]))
    return a


@pytest.mark.parametrize("change,status", BAD_DROPS + [
    (dict(rows=-1), "E_INVALID"), (dict(cols=-1), "E_INVALID"), (dict(cols=16385), "E_SIZE"), (dict(rows=2**31), "E_SIZE"),
    (dict(dtype=3), "E_INVALID"), (dict(gain_dtype=2), "E_INVALID"), (dict(x=None), "E_INVALID"), (dict(y=None), "E_INVALID"),
    (dict(gain=None), "E_INVALID"), (dict(gain=16386), "E_ALIGN"), (dict(x=4097), "E_ALIGN"), (dict(ld=299), "E_INVALID"), (dict(ld=2**41), "E_SIZE"),
    (dict(residual=64), "E_INVALID"), (dict(p=0.1), "E_INVALID"),                       # h has nowhere to go
    (dict(eps=-1.0), "E_INVALID"), (dict(eps=float("inf")), "E_INVALID"), (dict(eps=float("nan")), "E_INVALID"),
    (dict(rstd=2), "E_ALIGN"), (dict(y8=matrix(5, 300)), "E_INVALID"), (dict(y8=matrix(4, 299)), "E_INVALID"),
] + [(dict(y8=matrix(4, **c)), s) for c, s in BAD_MATRICES])
def test_refused_norm(change, status):
    a = norm_args(**change)
    refused(getattr(dopt, status), lambda: dopt._check(dopt._c["dopt_rms_norm"](ctypes.byref(a), None)))


def test_norm_of_nothing():
    for a in (norm_args(rows=0, x=None, y=None, gain=None), norm_args(cols=0, x=None, y=None, gain=None)):
        assert dopt._c["dopt_rms_norm"](ctypes.byref(a), None) == 0
    refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_rms_norm"](None, None)))
    refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_rms_norm_backward"](None, None, 0, None)))


@pytest.mark.parametrize("change,status", BAD_DROPS + [
    (dict(rows=-1), "E_INVALID"), (dict(cols=16385), "E_SIZE"), (dict(dtype=3), "E_INVALID"), (dict(gain=None), "E_INVALID"),
    (dict(dy=None), "E_INVALID"), (dict(h=None), "E_INVALID"), (dict(rstd=None), "E_INVALID"), (dict(rstd=6), "E_ALIGN"),
    (dict(dgain=6), "E_ALIGN"), (dict(dx=63), "E_ALIGN"),
    (dict(dh=None, dgain=None), "E_INVALID"), (dict(dy=4097), "E_ALIGN"), (dict(dres=3), "E_ALIGN"), (dict(ld=299), "E_INVALID"),
    (dict(ws=None), "E_INVALID"), (dict(ws=24), "E_ALIGN"), (dict(size=4 * 300 * 4 - 1), "E_SIZE")])
def test_refused_norm_backward(change, status):
    e = dict(rows=4, cols=300, dtype=1, gain_dtype=0, dy=4096, h=8192, dres=None, dh=12288, dx=None, gain=16384, rstd=32,
             dgain=64, p=0.0, d_step=None, ld=300, ws=1 << 20, size=1 << 20)
    e.update(change)
    r = [dopt.dopt_rows(e[k], e["ld"]) for k in ("dy", "h", "dres", "dh", "dx")]
    a = dopt.dopt_rms_norm_backward_args(e["rows"], e["cols"], e["dtype"], e["gain_dtype"], *r, e["gain"], e["rstd"],
                                         e["dgain"], 0, 0, dopt.dopt_drop(e["p"], 1, 2, 3, e["d_step"]))
    call = lambda: dopt._check(dopt._c["dopt_rms_norm_backward"](ctypes.byref(a), e["ws"], e["size"], None))  # noqa: E731
    refused(getattr(dopt, status), call)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_the_binding_refuses_what_the_pointers_would_hide():
    ok = dopt.Matrix8(u8(5, 48)[:, :40], u8(512))
    assert (ok.rows, ok.cols, ok.c.ld) == (5, 40, 48)
    for bad in ((torch.zeros(5, 48), u8(512)), (u8(5, 48).t(), u8(512)), (u8(5, 48), u8(511)), (u8(240), u8(512)),
                (u8(5, 1).expand(5, 48), u8(512)), (u8(5, 48), None), (u8(5, 48), torch.zeros(512)),
                (u8(1, 48).expand(5, 48), u8(512)), ([1], u8(512))):
        refused(dopt.E_INVALID, lambda: dopt.Matrix8(*bad))
    x = torch.zeros(5, 40)
    dopt.MatrixList([dict(values=x, out=ok)])
    for bad in (dict(values=x.double(), out=ok), dict(values=x[:, :39], out=ok), dict(values=x, out_t=ok),
                dict(values=x.t(), out=ok), dict(out=ok), dict(values=torch.zeros(200), out=ok)):
        refused(dopt.E_INVALID, lambda: dopt.MatrixList([bad]))
    drop = dopt.Dropout(0.1, -1, site=2, step=3)
    assert drop.c.seed == 0xFFFFFFFF
    refused(dopt.E_INVALID, lambda: dopt.Dropout(0.1, 1, d_step=torch.zeros(1)))
    for y, r in ((x.half(), None), (torch.zeros(5, 41), None), (x.t(), None), (x, x.half()), (None, None)):
        refused(dopt.E_INVALID, lambda: dopt.DropoutArgs(x, y, drop, residual=r))
    g = torch.ones(40)
    args = dopt.RmsNormArgs(x, g, 1e-6, y=x, dropout=drop, h=x)
    args.set_step(9)
    assert args.c.drop.step == 9 and drop.c.step == 3
    for kw in (dict(y=x.half()), dict(y=x[:4]), dict(y8=dopt.Matrix8(u8(5, 48), u8(512))), dict(y=x, rstd=torch.zeros(4)),
               dict(y=x, residual=x.half()), dict(y=x, h=torch.zeros(6, 40))):
        refused(dopt.E_INVALID, lambda: dopt.RmsNormArgs(x, g, 1e-6, **kw))
    refused(dopt.E_INVALID, lambda: dopt.RmsNormArgs(x, torch.ones(39), 1e-6, y=x))
    refused(dopt.E_INVALID, lambda: dopt.RmsNormArgs(x.half(), g.bfloat16(), 1e-6, y=x.half()))
    r = torch.zeros(5)
    for kw in (dict(dres=x.half()), dict(dgain=torch.zeros(40, dtype=torch.float16)), dict(dgain=torch.zeros(41)), dict(dx=x[:3])):
        refused(dopt.E_INVALID, lambda: dopt.RmsNormBackwardArgs(x, x, g, r, x, **kw))


def test_the_binding_refuses_host_memory():
    m, x, g = dopt.Matrix8(u8(5, 48)[:, :40], u8(512)), torch.zeros(5, 40), torch.ones(40)
    pairs = dopt.MatrixList([dict(values=x, out=m)])
    for call in (lambda: dopt.dopt_matrix8_pack(pairs), lambda: dopt.dopt_matrix8_unpack(pairs),
                 lambda: dopt.dopt_matrix8_multiply(m, m, torch.zeros(5, 5)),
                 lambda: dopt.dopt_dropout(dopt.DropoutArgs(x, x, dopt.Dropout(0.1, 1))),
                 lambda: dopt.dopt_rms_norm(dopt.RmsNormArgs(x, g, 1e-6, y=x)),
                 lambda: dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(x, x, g, torch.zeros(5), x))):
        assert "GPU" in refused(dopt.E_INVALID, call)
    for d in (torch.zeros(5, 6), torch.zeros(25), torch.zeros(5, 5, dtype=torch.int32), torch.zeros(5, 10)[:, ::2]):
        refused(dopt.E_INVALID, lambda: dopt.dopt_matrix8_multiply(m, m, d))


class OnGpu:
    """A stand-in for a torch tensor on a GPU of this index."""

    def __init__(self, index, *shape, dtype=torch.float32):
        self.index, self.shape, self.dtype = index, shape, dtype

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return int(np.prod(self.shape))

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1) if len(self.shape) == 2 else (1,)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index


def matrix_on(index):
    return dopt.Matrix8(OnGpu(index, 32, 48, dtype=torch.uint8), OnGpu(index, 512, dtype=torch.uint8))


def test_arrays_of_another_gpu_than_the_current(monkeypatch):
    """Every call is refused before a launch where one of its arrays is on another GPU than the current one: the
    launches, and the other arrays, are on that."""
    monkeypatch.setattr(dopt, "_current_device", lambda: 0)
    x0, x1, g0 = OnGpu(0, 32, 48), OnGpu(1, 32, 48), OnGpu(0, 48)
    d = lambda k: OnGpu(k, 32, 32)  # noqa: E731
    step = dopt.Dropout(0.1, 1, d_step=OnGpu(1, 1, dtype=torch.int64))
    r0, r1 = OnGpu(0, 32), OnGpu(1, 32)
    back = dict(workspace=OnGpu(1, 1 << 20, dtype=torch.uint8), workspace_bytes=1 << 20, dgain=g0)
    for call in (lambda: dopt.dopt_matrix8_multiply(matrix_on(1), matrix_on(1), d(1)),
                 lambda: dopt.dopt_matrix8_multiply(matrix_on(0), matrix_on(0), d(1)),
                 lambda: dopt.dopt_matrix8_multiply(matrix_on(0), matrix_on(1), d(0)),
                 lambda: dopt.dopt_matrix8_pack(dopt.MatrixList([dict(values=x1, out=matrix_on(0))])),
                 lambda: dopt.dopt_matrix8_unpack(dopt.MatrixList([dict(values=x1, out=matrix_on(1))])),
                 lambda: dopt.dopt_dropout(dopt.DropoutArgs(x1, x1, dopt.Dropout(0.1, 1))),
                 lambda: dopt.dopt_dropout(dopt.DropoutArgs(x0, x0, step)),
                 lambda: dopt.dopt_rms_norm(dopt.RmsNormArgs(x0, g0, 1e-6, y=x1)),
                 lambda: dopt.dopt_rms_norm(dopt.RmsNormArgs(x0, g0, 1e-6, y8=matrix_on(1))),
                 lambda: dopt.dopt_rms_norm(dopt.RmsNormArgs(x0, g0, 1e-6, y=x0, rstd=r1)),
                 lambda: dopt.dopt_rms_norm(dopt.RmsNormArgs(x0, g0, 1e-6, y=x0, h=x0, dropout=step)),
                 lambda: dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(x0, x1, g0, r0, x0)),
                 lambda: dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(x0, x0, g0, r0, x0, **back))):
        text = refused(dopt.E_INVALID, call)
        assert "GPU" in text


# -------------------------------------------------- the 64-bit restatement --

def test_places_are_a_permutation():
    for rows, cols in ((128, 512), (256, 1024), (128, 1500)):
        p = O.scale_places(rows, cols)
        assert len(np.unique(p)) == p.size and p.max() < O.scale_size(rows, cols)
    # 32 rows of 16 bytes: rows 0, 32, 64 and 96 of a tile side by side, four blocks each
    assert O.scale_places(128, 512)[[0, 32, 64, 96, 1]].tolist() == [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11], [12, 13, 14, 15], [16, 17, 18, 19]]


def test_rounding_is_to_the_nearest_value():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 200)) * np.exp(3 * rng.standard_normal((3, 200)))
    s = O.scales(x)
    got = O.rounded(x, s)
    for r in range(3):
        for c in range(200):
            v = np.concatenate([O.T.E4M3[:127], -O.T.E4M3[:127]]) * 2.0 ** (int(s[r, c // 128]) - 127)
            assert abs(got[r, c] - x[r, c]) == np.abs(v - x[r, c]).min()
    assert np.array_equal(O.scales(np.tile(x, (50, 1)), True)[:128], np.tile(O.scales(x).max(0), (128, 1)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_near_is_nearest_rounding(dtype):
    """Every value of a type is near what rounds to it, infinity too, and its neighbour's is not."""
    t = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[dtype]
    x = np.concatenate([np.geomspace(1e-9, 6e4, 5000), O.OVER[dtype] * np.array([0.999, 1 - 2.0**-20, 1, 1.5])])
    with np.errstate(over="ignore"):
        x = x.astype(np.float32).astype(np.float64)  # torch narrows by way of fp32
    got = torch.from_numpy(x).to(t).double().numpy()
    if dtype == "f32":
        got[-3] = x[-3] = torch.finfo(t).max
    assert np.isinf(got[-2:]).all() and np.isfinite(got[-4:-2]).all()
    assert O.near(got, x, 0.0, dtype).all() and O.near(-got, -x, 0.0, dtype).all()
    assert not O.near(-got, x, 0.0, dtype)[2000:].any()  # below that fp16 has subnormal numbers
    assert not O.near(got * (1 + 3 * O.EPS[dtype]), x, 0.0, dtype)[2000:-4].any()
    assert not O.near(np.full(2, torch.finfo(t).max), x[-2:], 0.0, dtype).any()


def test_random_numbers_are_the_steps():
    """The dropout's hash is that of the 8-bit moments' rounding."""
    r = O.random16(np.arange(1000), 5, 7, 11)
    assert np.array_equal(r, np.rint(O.T.rounding_fraction(1000, 7, 11, 5) * 65536))
    far = O.random16(np.array([0, 2**33, 2**34]), 5, 7, 11)
    assert len(set(far.tolist())) == 3
    share = (O.random16(np.arange(40000), 1, 2, 3) < O.threshold(0.1)).mean()
    assert abs(share - 0.1) < 6 * np.sqrt(0.09 / 40000)


def test_norm_backward_is_the_difference_quotient():
    rng = np.random.default_rng(2)
    h, gain, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    eps, step = 1e-3, 1e-6

    def loss(h, gain):
        return (O.norm(h, gain, eps)[1][0] * dy).sum()

    rstd = O.norm(h, gain, eps)[0][0]
    (dh, _), (dgain, _) = O.norm_backward(dy, h, gain, rstd, None)
    for r in range(3):
        for c in range(7):
            e = np.zeros_like(h)
            e[r, c] = step
            assert abs((loss(h + e, gain) - loss(h - e, gain)) / (2 * step) - dh[r, c]) < 1e-7
    for c in range(7):
        e = np.zeros_like(gain)
        e[c] = step
        assert abs((loss(h, gain + e) - loss(h, gain - e)) / (2 * step) - dgain[c]) < 1e-7
    assert np.allclose(O.norm_backward(dy, h, gain, rstd, dy)[0][0], dh + dy)
