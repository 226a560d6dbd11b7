"""Calls of the norm, its backward pass and dropout whose arrays share
elements, refused before any device work; and the arithmetic that finds them
against all pairs of elements."""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

from test_matrix8_host import dopt, drop_args, norm_args, refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_adam_gb300", "csrc")
ONE, SOME = "are one array", "share elements"
AT, LD, COLS = 1 << 20, 300, 200  # bytes; elements of 2 bytes, four rows


def backward_args(**kw):
    e = dict(dy=AT, h=2 * AT, dres=3 * AT, dh=4 * AT, dx=5 * AT)
    e.update(kw)
    r = [dopt.dopt_rows(e[k], e.get("ld_" + k, LD)) for k in ("dy", "h", "dres", "dh", "dx")]
    return dopt.dopt_rms_norm_backward_args(4, COLS, 1, 0, *r, 64, 32, None, 0, 0, dopt.dopt_drop(0.1, 1, 2, 3, None))


@pytest.mark.parametrize("change,text", [
    (dict(h=AT, y=AT), ONE), (dict(x=AT, h=AT, y=AT), ONE),
    (dict(h=AT, y=AT + 2), SOME), (dict(h=AT, y=AT + 600), SOME), (dict(h=AT + 3 * 600 + 398, y=AT), SOME), (dict(h=AT + 202, y=AT), SOME),
    (dict(x=AT, h=2 * AT, y=AT + 600), SOME), (dict(residual=AT, y=AT - 2, h=2 * AT), SOME), (dict(x=AT, h=AT + 2), SOME)])
def test_refused_norm(change, text):
    a = norm_args(**dict(dict(x=5 * AT, y=6 * AT, cols=COLS, ld=LD), **change))
    assert text in refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_rms_norm"](ctypes.byref(a), None)))


@pytest.mark.parametrize("change,text", [
    (dict(dh=AT, dx=AT), ONE), (dict(dh=7 * AT, dx=7 * AT), ONE), (dict(dh=7 * AT, dx=7 * AT, ld_dh=400), SOME),
    (dict(dh=7 * AT, dx=7 * AT + 600), SOME), (dict(dh=AT + 2), SOME), (dict(dx=2 * AT - 600), SOME), (dict(dx=3 * AT, ld_dx=250), SOME)])
def test_refused_norm_backward(change, text):
    a = backward_args(**change)
    assert text in refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_rms_norm_backward"](ctypes.byref(a), None, 0, None)))


@pytest.mark.parametrize("change", [dict(x=AT, y=AT + 2), dict(x=AT + 198, y=AT), dict(residual=AT + 2, y=AT), dict(x=AT, residual=AT, y=AT + 100)])
def test_refused_dropout(change):
    a = drop_args(**dict(dict(x=5 * AT, numel=100), **change))
    assert SOME in refused(dopt.E_INVALID, lambda: dopt._check(dopt._c["dopt_dropout"](ctypes.byref(a), None)))


def test_shared_elements_is_all_pairs(tmp_path):
    """shared_elements for small arrays at every kind of distance, against the elements themselves."""
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    rng = random.Random(1)
    cases, want = [], []
    for _ in range(4000):
        rows, cols, elem = rng.randint(1, 4), rng.randint(1, 5), rng.choice([2, 4])
        lda = cols + rng.randint(0, 4)
        ldb = lda if rng.random() < 0.8 else cols + rng.randint(0, 4)
        a, b = 4096, 4096 + elem * rng.choice([0, rng.randint(-30, 30)])
        at = [[{p + elem * (r * ld + c) for c in range(cols)} for r in range(rows)] for p, ld in ((a, lda), (b, ldb))]
        if at[0] == at[1]:
            w = 1
        elif rows > 1 and lda != ldb and a != b:
            w = 0  # not looked for
        else:
            w = 2 if set().union(*at[0]) & set().union(*at[1]) else 0
        cases.append((a, lda, b, ldb, rows, cols, elem))
        want.append(w)
    # far apart, and as many rows as there may be
    far = 1 << 42
    cases += [(far, 1 << 40, 2 * far, 1 << 40, 2**31 - 1, 16384, 4), (far, 1 << 40, far + 65536, 1 << 40, 2**31 - 1, 16384, 4),
              (far, 1 << 43, far - 4, 1 << 43, 1, 1 << 43, 4), (0, 8, 4096, 8, 4, 8, 4)]
    want += [2, 0, 2, 0]
    (tmp_path / "s.cpp").write_text(
        '#include <cstdio>\n#include "entry.h"\nint main() { long long a, la, b, lb, r, c, e;\n'
        'while (scanf("%lld %lld %lld %lld %lld %lld %lld", &a, &la, &b, &lb, &r, &c, &e) == 7)\n'
        'printf("%d\\n", (int)dopt::shared_elements((void*)a, la, (void*)b, lb, r, c, e)); }')
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.cpp"), "-o",
                    str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], input="\n".join(" ".join(map(str, c)) for c in cases), check=True, capture_output=True,
                         text=True).stdout.split()
    assert {0, 1, 2} == set(want) and list(map(int, out)) == want
