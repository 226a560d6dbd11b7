"""The binding of the step over a list of tensors without a GPU: which GPU's
memory a call may be given.  Every call here is refused before any launch: by
the library, for a negative learning rate, where the binding lets it through."""

import pytest
import torch

dopt = pytest.importorskip("mixed_precision_adam_gb300")
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
BAD = dict(HP, lr=-1.0)


def entry(**kw):
    """A valid bf16 tensor of pointers that are never followed."""
    e = dict(numel=1000, param=4096, grad=8192, master=12288, exp_avg=16384, exp_avg_sq=20480,
             param_dtype=dopt.BF16, grad_dtype=dopt.BF16)
    e.update(kw)
    return e


def refused(call):
    with pytest.raises(dopt.DoptError) as err:
        call()
    assert err.value.status == dopt.E_INVALID, err.value
    return str(err.value)


def refusal(lst):
    """Why a step with a bad learning rate is refused."""
    return refused(lambda: dopt.dopt_tensors_adam_step(lst, BAD, 1))


def test_good_grads_after_bad_ones():
    """A list given host grads is refused until it is given others, and no longer."""
    lst = dopt.TensorList([entry(), entry()])
    assert "hyper-parameters" in refusal(lst)
    lst.set_grads([torch.zeros(1000, dtype=torch.bfloat16), 8192])
    assert "GPU" in refusal(lst)
    lst.set_grads([8192, 8192])
    assert "hyper-parameters" in refusal(lst)
    # the other arrays' device stays
    lst = dopt.TensorList([entry(master=torch.zeros(1000))])
    lst.set_grads([8192])
    assert "GPU" in refusal(lst)


class OnGpu:
    """A stand-in for a torch tensor on a GPU of this index."""

    def __init__(self, index, numel=1000, dtype=torch.float32):
        self.index, self.n, self.dtype = index, numel, dtype

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.n

    @property
    def nbytes(self):
        return self.n * self.dtype.itemsize

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index


def on_gpu(index):
    return dict(param=OnGpu(index), grad=OnGpu(index), exp_avg=OnGpu(index), exp_avg_sq=OnGpu(index))


def test_lists_of_another_gpu_than_the_current(monkeypatch):
    """The launches go to the current device: a list of another one's memory is refused."""
    lst = dopt.TensorList([on_gpu(1)])
    moments = dict(exp_avg=OnGpu(1), exp_avg_codes=OnGpu(1, dtype=torch.uint8), exp_avg_scale=OnGpu(1, 4, torch.uint8))
    both = dopt.TensorList([on_gpu(1), on_gpu(0)])
    ws = dopt.dopt_tensors_workspace_bytes(1)
    monkeypatch.setattr(dopt, "_current_device", lambda: 0, raising=False)
    for call in (lambda: dopt.dopt_tensors_adam_step(lst, BAD, 1), lambda: dopt.dopt_tensors_step(lst, BAD, 1, 4096, ws),
                 lambda: dopt.dopt_tensors_grad_norm(lst, float("inf"), 1.0, 4096, ws, None, None, None),
                 lambda: dopt.dopt_state8_pack(dopt.MomentList([moments])),
                 lambda: dopt.dopt_state8_unpack(dopt.MomentList([moments]))):
        assert "GPU 1" in refused(call)
    monkeypatch.setattr(dopt, "_current_device", lambda: 1, raising=False)
    assert "hyper-parameters" in refusal(lst)
    assert "one GPU" in refusal(both)


def calls_with(lst, name, x):
    """Every call that takes the device argument `name`, each refused at the latest for its learning rate or loss
    scale."""
    ws = dopt.dopt_tensors_workspace_bytes(1)
    step = dict(workspace=4096, workspace_bytes=ws, d_step=None, d_lr=None, d_found_inf=None, d_norm=None)
    norm = dict(workspace=4096, workspace_bytes=ws, d_norm=None, d_clip_coef=None, d_found_inf=None)
    adam = dict(d_clip_coef=None, d_found_inf=None)
    out = []
    if name in step:
        out.append(lambda: dopt.dopt_tensors_step(lst, BAD, 1, **dict(step, **{name: x})))
    if name in norm:
        out.append(lambda: dopt.dopt_tensors_grad_norm(lst, float("inf"), 1.0, **dict(norm, **{name: x})))
    if name in adam:
        out.append(lambda: dopt.dopt_tensors_adam_step(lst, BAD, 1, **dict(adam, **{name: x})))
    return out


@pytest.mark.parametrize("name,dtype", [
    ("workspace", torch.uint8), ("d_step", torch.int64), ("d_lr", torch.float64), ("d_found_inf", torch.int32),
    ("d_norm", torch.float32), ("d_clip_coef", torch.float32)])
def test_device_arguments(monkeypatch, name, dtype):
    """The workspace and the scalars go to the kernels too: host memory, another GPU's, another type or fewer bytes
    are refused."""
    monkeypatch.setattr(dopt, "_current_device", lambda: 1, raising=False)
    lst = dopt.TensorList([entry()])
    need = dopt.dopt_tensors_workspace_bytes(1) if name == "workspace" else 1
    other = torch.bool if dtype != torch.uint8 else None
    for good in (4096, OnGpu(1, need, dtype), OnGpu(1, need * 8, torch.uint8)):
        for call in calls_with(lst, name, good):
            assert "hyper-parameters" in (text := refused(call)) or "inv_loss_scale" in text
    for bad, status in ((torch.zeros(need, dtype=dtype), dopt.E_INVALID), (torch.zeros(need, dtype=dtype).numpy(), dopt.E_INVALID),
                        (OnGpu(0, need, dtype), dopt.E_INVALID), (OnGpu(1, need, other), dopt.E_INVALID),
                        (OnGpu(1, need - 1, dtype), dopt.E_SIZE)):
        if getattr(bad, "dtype", 0) is None:
            continue
        for call in calls_with(lst, name, bad):
            with pytest.raises(dopt.DoptError) as err:
                call()
            assert err.value.status == status and name in str(err.value), err.value


@pytest.mark.parametrize("call", ["grad_norm", "adam_step", "step"])
def test_misaligned_scalars(call):
    """The kernels write and read the 4-byte scalars whole."""
    lst, ws = dopt.TensorList([entry()]), dopt.dopt_tensors_workspace_bytes(1)
    for at in (4097, 4098, 4099):
        for k in range(dict(grad_norm=3, adam_step=2, step=2)[call]):
            p = [at if j == k else None for j in range(3)]
            with pytest.raises(dopt.DoptError) as err:
                if call == "grad_norm":
                    dopt.dopt_tensors_grad_norm(lst, 1.0, 1.0, 4096, ws, *p)
                elif call == "adam_step":
                    dopt.dopt_tensors_adam_step(lst, HP, 1, d_clip_coef=p[0], d_found_inf=p[1])
                else:
                    dopt.dopt_tensors_step(lst, HP, 1, 4096, ws, d_found_inf=p[0], d_norm=p[1])
            assert err.value.status == dopt.E_ALIGN, err.value
