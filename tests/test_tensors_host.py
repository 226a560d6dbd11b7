"""The step over a list of tensors without a GPU: the struct layouts, the
refusals of every entry point (before any device work), and the 64-bit
restatement the GPU tests compare with, itself checked against brute force
and torch."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import tensors as O

dopt = pytest.importorskip("mixed_precision_adam_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
WS = 1 << 20


def entry(**kw):
    """A valid bf16 tensor of pointers that are never followed."""
    e = dict(numel=1000, param=4096, grad=8192, master=12288, exp_avg=16384, exp_avg_sq=20480,
             param_dtype=dopt.BF16, grad_dtype=dopt.BF16)
    e.update(kw)
    return e


def refused(status, call):
    with pytest.raises(dopt.DoptError) as err:
        call()
    assert err.value.status == status, err.value
    return str(err.value)


def calls(entries):
    lst = dopt.TensorList(entries)
    return [lambda: dopt.dopt_tensors_adam_step(lst, HP, 1),
            lambda: dopt.dopt_tensors_step(lst, HP, 1, 4096, WS)]


@pytest.mark.parametrize("name", ["dopt_tensor", "dopt_moment_tensor"])
def test_binding_structs_match_header(tmp_path, name):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    cls = getattr(dopt, name)
    body = "".join(f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_)
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dopt.h"\nint main(void) {'
                                  f'printf("size %zu\\n", sizeof({name}));{body}return 0;}}')
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    for line in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split("\n"):
        if line:
            field, value = line.split()
            assert (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset) == int(value), line


def test_sizes():
    assert [dopt.dopt_moment_blocks(n) for n in (0, 1, 256, 257, 2**40)] == [0, 1, 1, 2, 2**32]
    refused(dopt.E_INVALID, lambda: dopt.dopt_moment_blocks(-1))
    sizes = [dopt.dopt_tensors_workspace_bytes(n) for n in (0, 1, 1280, 1281, 10**6)]
    assert sizes[0] == sizes[1] == sizes[2] < sizes[3] < sizes[4] < 2**24
    refused(dopt.E_INVALID, lambda: dopt.dopt_tensors_workspace_bytes(-1))


@pytest.mark.parametrize("change,status", [
    (dict(numel=-1), "E_INVALID"), (dict(param_dtype=7), "E_INVALID"), (dict(grad_dtype=-1), "E_INVALID"),
    (dict(grad_dtype=2), "E_INVALID"),                      # fp16 grads of a bf16 param
    (dict(moments=2), "E_INVALID"), (dict(wd_mult=float("nan")), "E_INVALID"),
    (dict(param=None), "E_INVALID"), (dict(grad=None), "E_INVALID"), (dict(master=None), "E_INVALID"),
    (dict(exp_avg=None), "E_INVALID"), (dict(exp_avg_sq=None), "E_INVALID"),
    (dict(param_dtype=0, grad_dtype=0), "E_INVALID"),       # an fp32 param with a master
    (dict(param=4097), "E_ALIGN"), (dict(grad=8193), "E_ALIGN"), (dict(master=12290), "E_ALIGN"),
    (dict(exp_avg=16386), "E_ALIGN"), (dict(exp_avg_sq=20481), "E_ALIGN"),
    (dict(moments=1), "E_INVALID"),                         # 8-bit moments without scales
    (dict(moments=1, exp_avg_scale=64), "E_INVALID"),
    (dict(moments=0, exp_avg_scale=64, exp_avg_sq_scale=64), "E_INVALID"),
    (dict(numel=2**50), "E_SIZE"),
])
def test_refused_tensors(change, status):
    for call in calls([entry(), entry(**change)]):
        assert "tensor 1" in refused(getattr(dopt, status), call)


def test_refused_arguments():
    lst = dopt.TensorList([entry()])
    for bad in (dict(lr=-1.0), dict(lr=float("inf")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0),
                dict(weight_decay=float("nan"))):
        for call in (lambda: dopt.dopt_tensors_adam_step(lst, dict(HP, **bad), 1),
                     lambda: dopt.dopt_tensors_step(lst, dict(HP, **bad), 1, 4096, WS)):
            refused(dopt.E_INVALID, call)
    refused(dopt.E_INVALID, lambda: dopt.dopt_tensors_adam_step(lst, HP, 0))
    refused(dopt.E_INVALID, lambda: dopt.dopt_tensors_adam_step(lst, HP, 1, float("nan")))
    need = dopt.dopt_tensors_workspace_bytes(1)

    def norm(inv=1.0, max_norm=1.0, ws=4096, size=need):
        return lambda: dopt.dopt_tensors_grad_norm(lst, inv, max_norm, ws, size, None, None, None)

    for call, status in ((norm(inv=float("inf")), dopt.E_INVALID), (norm(max_norm=float("nan")), dopt.E_INVALID),
                         (norm(ws=None), dopt.E_INVALID), (norm(ws=4100), dopt.E_ALIGN), (norm(size=need - 1), dopt.E_SIZE),
                         (lambda: dopt.dopt_tensors_step(lst, HP, 1, 4096, need - 1), dopt.E_SIZE),
                         (lambda: dopt.dopt_tensors_step(lst, HP, 1, 4096, need, d_step=12), dopt.E_ALIGN),
                         (lambda: dopt.dopt_tensors_step(lst, HP, 1, 4096, need, d_step=16, d_lr=20), dopt.E_ALIGN)):
        refused(status, call)
    refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_tensors_adam_step"](None, 1, None, 1.0, 0, None, None, None)))
    refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_tensors_adam_step"](lst.c, 1, None, 1.0, 0, None, None, None)))
    refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_tensors_adam_step"](lst.c, -1, None, 1.0, 0, None, None, None)))


@pytest.mark.parametrize("change,status", [
    (dict(numel=-1), "E_INVALID"), (dict(values_dtype=dopt.F16), "E_INVALID"), (dict(exp_avg=6), "E_ALIGN"),
    (dict(exp_avg_codes=None), "E_INVALID"), (dict(exp_avg_sq_scale=None), "E_INVALID"), (dict(numel=2**50), "E_SIZE"),
])
def test_refused_moments(change, status):
    e = dict(numel=100, exp_avg=64, exp_avg_sq=128, exp_avg_codes=3, exp_avg_sq_codes=5, exp_avg_scale=7,
             exp_avg_sq_scale=9)
    lst = dopt.MomentList([dict(e, **change)])
    for fn in (dopt.dopt_state8_pack, dopt.dopt_state8_unpack):
        refused(getattr(dopt, status), lambda: fn(lst))


def test_the_binding_refuses_what_the_pointers_would_hide():
    x = torch.zeros(4, 6)
    ok = dict(param=torch.zeros(24), grad=torch.zeros(24), exp_avg=torch.zeros(24), exp_avg_sq=torch.zeros(24))
    dopt.TensorList([ok])
    eight = dict(ok, exp_avg=torch.zeros(24, dtype=torch.uint8), exp_avg_sq=torch.zeros(24, dtype=torch.uint8))
    for bad in (dict(ok, grad=x.t()), dict(ok, param=torch.zeros(48)[::2]), dict(ok, grad=torch.zeros(23)),
                dict(ok, exp_avg=torch.zeros(24, dtype=torch.float64)), dict(ok, exp_avg=eight["exp_avg"]), eight,
                dict(eight, exp_avg_scale=torch.zeros(2, dtype=torch.uint8), exp_avg_sq_scale=torch.zeros(1, dtype=torch.uint8)),
                dict(ok, grad=torch.zeros(24, dtype=torch.int32))):
        refused(dopt.E_INVALID, lambda: dopt.TensorList([bad]))
    lst = dopt.TensorList([ok])
    lst.set_grads([x.view(-1)])
    assert lst.c[0].grad == x.data_ptr()
    for bad in ([], [x.t()], [torch.zeros(23)], [torch.zeros(24, dtype=torch.float16)]):
        refused(dopt.E_INVALID, lambda: lst.set_grads(bad))
    assert lst.c[0].grad == x.data_ptr()  # a refused change leaves the list as it was
    m = dict(exp_avg=torch.zeros(24), exp_avg_codes=torch.zeros(24, dtype=torch.uint8),
             exp_avg_scale=torch.zeros(1, dtype=torch.uint8))
    dopt.MomentList([m])
    for bad in (dict(m, exp_avg=torch.zeros(24, dtype=torch.float16)), dict(m, exp_avg_codes=torch.zeros(24)),
                dict(m, exp_avg_sq=torch.zeros(24, dtype=torch.bfloat16)), dict()):
        refused(dopt.E_INVALID, lambda: dopt.MomentList([bad]))


def test_the_binding_refuses_host_memory():
    """Lists may be made of CPU tensors, but no kernel gets their addresses."""
    ok = dict(param=torch.zeros(24), grad=torch.zeros(24), exp_avg=torch.zeros(24), exp_avg_sq=torch.zeros(24))
    lst = dopt.TensorList([ok])
    ws = dopt.dopt_tensors_workspace_bytes(1)
    for call in (lambda: dopt.dopt_tensors_adam_step(lst, HP, 1), lambda: dopt.dopt_tensors_step(lst, HP, 1, 4096, ws),
                 lambda: dopt.dopt_tensors_grad_norm(lst, 1.0, 1.0, 4096, ws, None, None, None)):
        refused(dopt.E_INVALID, call)
    m = dict(exp_avg=torch.zeros(24), exp_avg_codes=torch.zeros(24, dtype=torch.uint8),
             exp_avg_scale=torch.zeros(1, dtype=torch.uint8))
    for fn in (dopt.dopt_state8_pack, dopt.dopt_state8_unpack):
        refused(dopt.E_INVALID, lambda: fn(dopt.MomentList([m])))
    refused(dopt.E_INVALID, lambda: dopt.TensorList([dict(ok, grad=np.zeros(24, np.float32))]))
    lst = dopt.TensorList([entry()])
    lst.set_grads([torch.zeros(1000, dtype=torch.bfloat16)])
    refused(dopt.E_INVALID, lambda: dopt.dopt_tensors_adam_step(lst, HP, 1))
    refused(dopt.E_INVALID, lambda: dopt.TensorList([dict(ok, moments=dopt.MOMENTS_8BIT)]))


# -------------------------------------------------- the 64-bit restatement --

def test_e4m3_values_are_torchs():
    codes = torch.arange(256).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = O.m_values(np.repeat(codes.numpy(), 256).reshape(256, 256).T.reshape(-1), np.full(256, 127))[:256]
    assert np.array_equal(got, want, equal_nan=True)


def test_rounding_is_to_the_nearest_value():
    """Against all the values there are, by brute force."""
    rng = np.random.default_rng(1)
    m = rng.standard_normal(512) * np.exp(3 * rng.standard_normal(512))
    s = O.m_scale(m)
    got = O.m_rounded(m, s)
    for i in range(512):
        values = np.concatenate([O.E4M3[:127], -O.E4M3[:127]]) * 2.0 ** (int(s[i // 256]) - 127)
        assert abs(got[i] - m[i]) == np.abs(values - m[i]).min()
    v = m * m
    s = O.v_scale(v)
    got = O.v_rounded(v, s, 0.5)
    for i in range(512):
        values = O.v_values(np.arange(256), [s[i // 256]])[1:]
        assert abs(got[i] - v[i]) == np.abs(values - v[i]).min()


@pytest.mark.parametrize("top,want_m,want_v", [
    (448.0, 127, 104), (448.1, 128, 104), (480.0, 128, 104), (480.1, 128, 105), (1.0, 119, 96), (0.0, 8, 0),
    (np.inf, 255, 255), (np.nan, 255, 255), (2.0**-149, 8, 0), (3.4e38, 255, 255), (1.75 * 2.0**127, 246, 223),
])
def test_scales(top, want_m, want_v):
    x = np.zeros(300)
    x[7] = top
    assert O.m_scale(x).tolist() == [want_m, 8] and O.v_scale(x).tolist() == [want_v, 0]
    if want_m != 255 and top >= 1:  # the largest value keeps a code within half of the last place
        assert abs(O.m_rounded(x, O.m_scale(x))[7] - top) <= top / 16 and abs(O.v_rounded(x, O.v_scale(x), 0.5)[7] - top) <= top / 16


def test_rounding_bits_are_spread():
    """65,536 elements of 3 steps: each of 16 bins near its share, neighbours and steps unrelated (6 standard
    errors)."""
    f = [O.rounding_fraction(65536, 3, t, 77) for t in (1, 2, 3)]
    for x in f:
        assert np.abs(np.histogram(x, 16, (0, 1))[0] - 4096).max() < 6 * 64
        assert abs(np.corrcoef(x[:-1], x[1:])[0, 1]) < 6 / 256
    assert abs(np.corrcoef(f[0], f[1])[0, 1]) < 6 / 256 and abs(np.corrcoef(f[1], f[2])[0, 1]) < 6 / 256
    assert np.array_equal(O.rounding_fraction(100, 3, 1, 77, first=1001), f[0][1001:1101])


def test_adamw_is_torchs():
    rng = np.random.default_rng(2)
    w, g = rng.standard_normal(100), rng.standard_normal((3, 100))
    p = torch.nn.Parameter(torch.from_numpy(w.copy()))
    opt = torch.optim.AdamW([p], lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m = v = np.zeros(100)
    for t in range(1, 4):
        p.grad = torch.from_numpy(g[t - 1] * 0.25 * 0.5)
        opt.step()
        (w, m, v), _ = O.adamw(w, g[t - 1], m, v, HP, t, 0.25, 0.5)
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-13)


def test_grad_norm_is_torchs():
    gs = [torch.randn(50, dtype=torch.float64), torch.randn(3, 7, dtype=torch.float64)]
    ps = [torch.nn.Parameter(torch.zeros_like(g)) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = g.clone()
    norm = torch.nn.utils.clip_grad_norm_(ps, 0.5)
    got = O.grad_norm([g.numpy() for g in gs], 1.0, 0.5)
    assert abs(got[0] - norm.item()) < 1e-12
    assert abs(ps[0].grad[0].item() - gs[0][0].item() * got[1]) < 1e-12
