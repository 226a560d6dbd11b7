"""The binding of the step over a list of tensors without a GPU: which GPU's
memory a call may be given.  Every call here is refused before any launch: a
step number of 0 is, by the library, where the binding lets a call through."""

import pytest
import torch

dopt = pytest.importorskip("mixed_precision_adam_gb300")
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


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
    """Why a step of step number 0 is refused."""
    return refused(lambda: dopt.dopt_tensors_adam_step(lst, HP, 0))


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

    def element_size(self):
        return self.dtype.itemsize

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
    for call in (lambda: dopt.dopt_tensors_adam_step(lst, HP, 1), lambda: dopt.dopt_tensors_step(lst, HP, 1, 4096, ws),
                 lambda: dopt.dopt_tensors_grad_norm(lst, 1.0, 1.0, 4096, ws, None, None, None),
                 lambda: dopt.dopt_state8_pack(dopt.MomentList([moments])),
                 lambda: dopt.dopt_state8_unpack(dopt.MomentList([moments]))):
        assert "GPU 1" in refused(call)
    monkeypatch.setattr(dopt, "_current_device", lambda: 1, raising=False)
    assert "hyper-parameters" in refusal(lst)
    assert "one GPU" in refusal(both)
