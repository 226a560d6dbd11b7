"""The README's lines for the step over a list of tensors run as they stand,
and every step takes the grads of its own backward pass."""

import os
import textwrap

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_lines():
    text = open(os.path.join(ROOT, "README.md")).read()
    at = text.index("    params = [p for p in model.parameters()]")
    lines = text[at:].split("\n")
    end = next(i for i, line in enumerate(lines) if line and not line.startswith("    "))
    return textwrap.dedent("\n".join(lines[:end]))


def test_readme_list_step():
    torch.manual_seed(1)
    model = torch.nn.Sequential(torch.nn.Linear(300, 70), torch.nn.Tanh(), torch.nn.Linear(70, 9)).cuda().bfloat16()
    data = [(torch.randn(32, 300, device="cuda").bfloat16(), torch.randn(32, 9, device="cuda").bfloat16()) for _ in range(4)]
    used = []
    real = dopt.dopt_tensors_step

    def step(tensors, *a, **kw):
        real(tensors, *a, **kw)
        used.append([(tensors.c[k].grad, p.grad.data_ptr()) for k, p in enumerate(model.parameters())])

    class Dopt:
        TensorList, dopt_tensors_step = dopt.TensorList, staticmethod(step)
        dopt_moment_blocks = staticmethod(dopt.dopt_moment_blocks)
        dopt_tensors_workspace_bytes = staticmethod(dopt.dopt_tensors_workspace_bytes)

    scope = dict(torch=torch, dopt=Dopt, model=model, batches=data, loss_fn=torch.nn.functional.mse_loss,
                 hp=dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1))
    before = [p.detach().clone() for p in model.parameters()]
    exec(readme_lines(), scope)
    assert len(used) == 4 and all(a == b for pairs in used for a, b in pairs)
    assert int(scope["applied"]) == 4
    for p, b in zip(model.parameters(), before):
        assert torch.isfinite(p).all() and not torch.equal(p, b)
