"""Training a small model with the optimizer step over a list of tensors.

    python examples/tensor_list_step.py                 # 8-bit moments
    python examples/tensor_list_step.py --moments 32    # fp32 moments
    python examples/tensor_list_step.py --matrices 8    # 8-bit products, dropout on the blocks' branches

A bf16 residual MLP with fp32 gains learns a fixed random function.  The
list holds every parameter: matrices with an fp32 master copy, gains stepped
in place and not decayed.  Each training step is one call: the grads' global
norm, the clip, the skip of a step with a non-finite grad, and AdamW, all on
the device; the step number lives there too, so nothing waits for the GPU.
Halfway the 8-bit moments go through a checkpoint: unpacked to bf16 values
(exact), packed again.

With --matrices 8 the blocks compute with the library too: dropout, the
residual's addition and the RMS norm in one call, products of 8-bit matrices
forward and backward, and the weights packed again after each step.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_adam_gb300 as dopt  # noqa: E402

HP = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01)


class Block(torch.nn.Module):
    def __init__(self, d):
        super().__init__()
        self.gain = torch.nn.Parameter(torch.ones(d))
        self.up = torch.nn.Linear(d, 2 * d, bias=False)
        self.down = torch.nn.Linear(2 * d, d, bias=False)

    def forward(self, x):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * self.gain
        return x + self.down(torch.nn.functional.silu(self.up(y.to(x.dtype))))


def stream():
    return torch.cuda.current_stream()


def matrix8(rows, cols):
    """An 8-bit matrix's memory: rows of codes on 16-byte boundaries, and scales."""
    codes = torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda")[:, :cols]
    return dopt.Matrix8(codes, torch.empty(dopt.dopt_matrix8_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda"))


def packed(x):
    """x (rows of tokens) and its transpose, packed in one pass."""
    out, out_t = matrix8(*x.shape), matrix8(*x.shape[::-1])
    dopt.dopt_matrix8_pack(dopt.MatrixList([dict(values=x, out=out, out_t=out_t)]), stream=stream())
    return out, out_t


class Product8(torch.autograd.Function):
    """x w^T of 8-bit matrices; w and its transpose are packed in squares, which both read the same."""

    @staticmethod
    def forward(ctx, x, weight, w8, w8_t):
        x8, x8_t = packed(x)
        y = torch.empty(x.shape[0], weight.shape[0], dtype=x.dtype, device="cuda")
        dopt.dopt_matrix8_multiply(x8, w8, y, stream=stream())
        ctx.x8_t, ctx.w8_t, ctx.weight = x8_t, w8_t, weight
        return y

    @staticmethod
    def backward(ctx, dy):
        dy8, dy8_t = packed(dy.contiguous())
        dx = torch.empty(dy.shape[0], ctx.weight.shape[1], dtype=dy.dtype, device="cuda")
        dopt.dopt_matrix8_multiply(dy8, ctx.w8_t, dx, stream=stream())
        dw = torch.empty(ctx.weight.shape, dtype=ctx.weight.dtype, device="cuda")
        dopt.dopt_matrix8_multiply(dy8_t, ctx.x8_t, dw, stream=stream())
        return dx, dw, None, None


class Norm8(torch.autograd.Function):
    """(h, norm of h) with h = dropout(branch) + x, or (x, norm of x) without a branch."""

    @staticmethod
    def forward(ctx, x, branch, gain, drop):
        rows, cols = x.shape
        h = x if branch is None else torch.empty_like(x)
        y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
        source = dict(x=x) if branch is None else dict(x=branch, residual=x, h=h, dropout=drop)
        dopt.dopt_rms_norm(dopt.RmsNormArgs(gain=gain.detach(), eps=1e-6, y=y, rstd=rstd, **source), stream=stream())
        ctx.save_for_backward(h, gain, rstd)
        ctx.branch, ctx.drop = branch is not None, drop
        return h.view_as(h), y

    @staticmethod
    def backward(ctx, dh_after, dy):
        h, gain, rstd = ctx.saved_tensors
        dh, dgain = torch.empty_like(h), torch.empty_like(gain)
        dx = torch.empty_like(h) if ctx.branch else None
        size = dopt.dopt_rms_norm_workspace_bytes(*h.shape)
        dopt.dopt_rms_norm_backward(dopt.RmsNormBackwardArgs(
            dy.contiguous(), h, gain.detach(), rstd, dh, dres=dh_after.contiguous(), dx=dx, dropout=ctx.drop if ctx.branch else None,
            dgain=dgain, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"), workspace_bytes=size), stream=stream())
        return dh, dx, dgain, None


class Model8(torch.nn.Module):
    """build_model's Sequential, its blocks computed by the library: a block's branch is added, with dropout, by the
    next block's norm."""

    def __init__(self, model, p, applied):
        super().__init__()
        self.first, self.blocks, self.last = model[0], torch.nn.ModuleList(model[1:-1]), model[-1]
        self.p, self.applied = p, applied  # the steps so far, on the device: each step has other masks
        self.weights = {m: (matrix8(*m.weight.shape), matrix8(*m.weight.shape[::-1]))
                        for b in self.blocks for m in (b.up, b.down)}
        self.pack_list = dopt.MatrixList([dict(values=m.weight.data, block=dopt.BLOCK_SQUARE, out=w, out_t=w_t)
                                          for m, (w, w_t) in self.weights.items()])

    def pack_weights(self):
        dopt.dopt_matrix8_pack(self.pack_list, stream=stream())

    def forward(self, x):
        h, branch = self.first(x), None
        for k, b in enumerate(self.blocks):
            drop = dopt.Dropout(self.p, 7, site=k, d_step=self.applied) if k else None
            h, y = Norm8.apply(h, branch, b.gain, drop)
            y = torch.nn.functional.silu(Product8.apply(y, b.up.weight, *self.weights[b.up]))
            branch = Product8.apply(y, b.down.weight, *self.weights[b.down])
        return self.last(h + branch)


def build_model(d, layers, dtype, seed):
    torch.manual_seed(seed)
    model = torch.nn.Sequential(torch.nn.Linear(d, d, bias=False), *[Block(d) for _ in range(layers)],
                                torch.nn.Linear(d, d, bias=False)).cuda()
    for p in model.parameters():
        if p.dim() > 1:
            p.data = p.data.to(dtype)
    return model


class Optimizer:
    """The state of one TensorList and its step."""

    def __init__(self, params, moments):
        self.params, self.moments, entries = list(params), moments, []
        for p in self.params:
            n = p.numel()
            e = dict(param=p.data, grad=torch.zeros_like(p.data), wd_mult=1.0 if p.dim() > 1 else 0.0)
            if p.dtype != torch.float32:
                e["master"] = p.data.float()
            for name in ("exp_avg", "exp_avg_sq"):
                e[name] = torch.zeros(n, dtype=torch.uint8 if moments == 8 else torch.float32, device="cuda")
                if moments == 8:
                    e[name + "_scale"] = torch.zeros(dopt.dopt_moment_blocks(n), dtype=torch.uint8, device="cuda")
            entries.append(e)
        self.entries = entries
        self.list = dopt.TensorList(entries)
        self.workspace = torch.empty(dopt.dopt_tensors_workspace_bytes(self.list.n), dtype=torch.uint8, device="cuda")
        self.applied = torch.zeros(1, dtype=torch.int64, device="cuda")  # steps so far

    def step(self, inv_loss_scale=1.0, max_norm=1.0):
        self.list.set_grads([p.grad for p in self.params])
        dopt.dopt_tensors_step(self.list, HP, 1, self.workspace, self.workspace.numel(),
                               inv_loss_scale=inv_loss_scale, max_norm=max_norm, seed=1, d_step=self.applied,
                               stream=torch.cuda.current_stream())

    def moment_values(self, dtype=torch.bfloat16):
        """The moments as values, by parameter (of 8-bit ones: unpacked, exactly)."""
        if self.moments == 32:
            return [dict(exp_avg=e["exp_avg"], exp_avg_sq=e["exp_avg_sq"]) for e in self.entries]
        out = [{k: torch.empty(e[k].numel(), dtype=dtype, device="cuda") for k in ("exp_avg", "exp_avg_sq")}
               for e in self.entries]
        dopt.dopt_state8_unpack(self._moment_list(out), stream=torch.cuda.current_stream())
        return out

    def load_moment_values(self, values):
        if self.moments == 32:
            for e, v in zip(self.entries, values):
                e["exp_avg"].copy_(v["exp_avg"])
                e["exp_avg_sq"].copy_(v["exp_avg_sq"])
        else:
            dopt.dopt_state8_pack(self._moment_list(values), stream=torch.cuda.current_stream())

    def _moment_list(self, values):
        return dopt.MomentList([dict(v, exp_avg_codes=e["exp_avg"], exp_avg_sq_codes=e["exp_avg_sq"],
                                     exp_avg_scale=e["exp_avg_scale"], exp_avg_sq_scale=e["exp_avg_sq_scale"])
                                for e, v in zip(self.entries, values)])


def train(moments=8, steps=200, d=256, layers=4, batch=1024, matrices=16, p=0.05):
    """Returns the losses, the grad norm of the last step and the number of applied steps."""
    teacher = build_model(d, 1, torch.bfloat16, seed=1)
    model = build_model(d, layers, torch.bfloat16, seed=2)
    opt = Optimizer(model.parameters(), moments)
    if matrices == 8:
        model = Model8(model, p, opt.applied)
    gen = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for t in range(steps):
        x = torch.randn(batch, d, generator=gen, device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            y = teacher(x)
        if matrices == 8:
            model.pack_weights()
        loss = (model(x).float() - y.float()).square().mean()
        model.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if t == steps // 2:
            opt.load_moment_values(opt.moment_values())
    stats = dopt.dopt_read_step_stats(opt.workspace, torch.cuda.current_stream())
    return torch.stack(losses).tolist(), stats["grad_norm"], int(opt.applied)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--moments", type=int, choices=(8, 32), default=8)
    ap.add_argument("--matrices", type=int, choices=(8, 16), default=16)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    losses, norm, applied = train(a.moments, a.steps, matrices=a.matrices)
    for t in list(range(0, a.steps, max(1, a.steps // 10))) + [a.steps - 1]:
        print(f"step {t + 1}: loss {losses[t]:.5f}")
    print(f"{applied} steps applied, the last grad norm {norm:.4f}, {a.moments}-bit moments, {a.matrices}-bit matrices")
