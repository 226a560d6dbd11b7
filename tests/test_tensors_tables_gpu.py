"""The step over a list of tensors around what one launch holds: the tensors of
a table (40 and 360 in AdamW, 60 and 500 in pack and unpack, one table for
each values type), and the tiles of a CTA's walk."""

import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from oracle import tensors as O  # noqa: E402
from tests.tensors_harness import TORCH, Array, Case  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECKED = os.path.join(ROOT, "mixed_precision_adam_gb300", "lib", "libdopt_checked.so")


@pytest.mark.parametrize("count", [359, 360, 361, 720, 721])
@pytest.mark.parametrize("moments", [32, 8])
def test_step_of_full_tables(count, moments):
    case = Case([dict(numel=1 + (k * 37) % 300, param="bf16", grad="bf16", moments=moments) for k in range(count)], seed=6)
    for step in (3, 4):
        dopt.dopt_tensors_adam_step(case.list, dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1), step, 1.0, 1)
        case.check_step(step, seed=1)


@pytest.mark.parametrize("count", [59, 60, 61, 499, 500, 501, 1001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack_and_unpack_of_full_tables(count, dtype):
    """One values type, so that the counts are those of its tables; both moments, their scales, and the way back."""
    gen = torch.Generator().manual_seed(count)
    cases = []
    for k in range(count):
        n = 1 + (k * 29) % 300
        size = torch.exp(torch.randn(n, generator=gen) * 3) * 1e-4
        a = dict(exp_avg=Array(torch.randn(n, generator=gen) * size, TORCH[dtype]),
                 exp_avg_sq=Array(torch.rand(n, generator=gen) * size * size, TORCH[dtype]))
        for name in ("exp_avg", "exp_avg_sq"):
            a[name + "_codes"] = Array(torch.zeros(n), torch.uint8)
            a[name + "_scale"] = Array(torch.zeros(-(-n // 256)), torch.uint8)
        cases.append(a)
    lst = dopt.MomentList([{k: x.view for k, x in a.items()} for a in cases])
    dopt.dopt_state8_pack(lst)
    torch.cuda.synchronize()
    packed = [{k: x.numpy() for k, x in a.items()} for a in cases]
    for k, b in enumerate(packed):
        m, v = b["exp_avg"].astype(np.float64), b["exp_avg_sq"].astype(np.float64)
        assert np.array_equal(b["exp_avg_scale"], O.m_scale(m)) and np.array_equal(b["exp_avg_sq_scale"], O.v_scale(v)), k
        assert np.array_equal(O.m_values(b["exp_avg_codes"], b["exp_avg_scale"]), O.m_rounded(m, b["exp_avg_scale"])), k
        assert np.array_equal(O.v_values(b["exp_avg_sq_codes"], b["exp_avg_sq_scale"]),
                              O.v_rounded(v, b["exp_avg_sq_scale"], 0.5)), k
    dopt.dopt_state8_unpack(lst)
    torch.cuda.synchronize()
    for k, (a, b) in enumerate(zip(cases, packed)):
        assert np.array_equal(a["exp_avg"].numpy(), O.m_values(b["exp_avg_codes"], b["exp_avg_scale"])), k
        assert np.array_equal(a["exp_avg_sq"].numpy(), O.v_values(b["exp_avg_sq_codes"], b["exp_avg_sq_scale"])), k
        assert all(x.guards_intact() for x in a.values()), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack_and_unpack_of_several_walks(dtype):
    """Past what the resident CTAs walk over at first (5e6 elements in unpack, 2.5e7 in pack): one tensor, and
    small ones behind it, against the same in pieces that a single walk covers, and windows against the
    restatement."""
    gen = torch.Generator(device="cuda").manual_seed(19)
    sizes = [60_000_321, 700, 1, 5000]
    piece = 4_000_000 // 256 * 256

    def moments(n):
        size = torch.exp(torch.randn(n, generator=gen, device="cuda") * 3) * 1e-4
        return dict(exp_avg=(torch.randn(n, generator=gen, device="cuda") * size).to(TORCH[dtype]),
                    exp_avg_sq=(torch.rand(n, generator=gen, device="cuda") * size * size).to(TORCH[dtype]))

    def codes(n):
        return {name + end: torch.full((n if end == "_codes" else -(-n // 256),), 77, dtype=torch.uint8, device="cuda")
                for name in ("exp_avg", "exp_avg_sq") for end in ("_codes", "_scale")}

    values = [moments(n) for n in sizes]
    whole, parts = [codes(n) for n in sizes], [codes(n) for n in sizes]
    dopt.dopt_state8_pack(dopt.MomentList([dict(v, **c) for v, c in zip(values, whole)]))
    back = [{k: torch.full_like(x, 77) for k, x in v.items()} for v in values]
    dopt.dopt_state8_unpack(dopt.MomentList([dict(b, **c) for b, c in zip(back, whole)]))
    pieces = [{k: torch.full_like(x, 77) for k, x in v.items()} for v in values]
    for v, c, p in zip(values, parts, pieces):
        for at in range(0, v["exp_avg"].numel(), piece):
            def cut(d, at=at):
                return {k: x[at // 256: (at + piece) // 256] if k.endswith("_scale") else x[at:at + piece] for k, x in d.items()}
            dopt.dopt_state8_pack(dopt.MomentList([dict(cut(v), **cut(c))]))
            dopt.dopt_state8_unpack(dopt.MomentList([dict(cut(p), **cut(c))]))
    torch.cuda.synchronize()
    for k in range(len(sizes)):
        for name in whole[k]:
            assert torch.equal(whole[k][name], parts[k][name]), (k, name)
        for name in back[k]:
            assert torch.equal(back[k][name], pieces[k][name]), (k, name)
    n = sizes[0]
    for at, end in ((0, 4096), (24_903_680 - 2048, 24_903_680 + 2048), (n // 256 * 256 - 4096, n)):
        b = {k: x[at // 256: -(-end // 256)] if k.endswith("_scale") else x[at:end] for k, x in whole[0].items()}
        b = {k: x.cpu().numpy() for k, x in b.items()}
        m, v = (values[0][k][at:end].double().cpu().numpy() for k in ("exp_avg", "exp_avg_sq"))
        assert np.array_equal(O.m_values(b["exp_avg_codes"], b["exp_avg_scale"]), O.m_rounded(m, O.m_scale(m)))
        assert np.array_equal(O.v_values(b["exp_avg_sq_codes"], b["exp_avg_sq_scale"]), O.v_rounded(v, O.v_scale(v), 0.5))
        assert np.array_equal(back[0]["exp_avg"][at:end].double().cpu().numpy(), O.m_rounded(m, O.m_scale(m)))


@pytest.mark.skipif("libdopt_checked" in os.environ.get("DOPT_LIBRARY", ""), reason="already the checked build")
def test_edges_and_tables_under_the_bounds_checked_build():
    assert os.path.exists(CHECKED)
    files = [os.path.join(ROOT, "tests", f) for f in ("test_tensors_edges_gpu.py", "test_tensors_tables_gpu.py")]
    out = subprocess.run([sys.executable, "-m", "pytest", *files, "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=dict(os.environ, DOPT_LIBRARY=CHECKED), capture_output=True, text=True, timeout=900)
    assert out.returncode == 0, out.stdout[-4000:] + out.stderr[-2000:]
    assert " passed" in out.stdout
