"""The training-side calls refuse tensors that are not on the GPU, before anything reaches it: first with every tensor in
host memory (no GPU needed), then with one of them there beside others on the GPU."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg

BF16 = torch.bfloat16


def operands(device):
    e = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=device)
    f = dict(dtype=torch.float32)
    head = dict(X=e(8, 64), W=e(100, 64), labels=e(8, dtype=torch.int64))
    return {
        tkg.linear_ce_loss: dict(head, loss=e(8, **f), lse=e(8, **f)),
        tkg.linear_ce_grad: dict(head, lse=e(8, **f), dloss=e(8, **f), dX=e(8, 64), dW=e(100, 64)),
        tkg.gemm_grouped_dev_bf16_dgrad: dict(sizes_dev=e(2, dtype=torch.int32), dD=e(30, 64), B=e(2, 64, 128),
                                              dA=e(30, 128)),
        tkg.gemm_grouped_dev_bf16_wgrad: dict(sizes_dev=e(2, dtype=torch.int32), dD=e(30, 64), A=e(30, 128),
                                              dB=e(2, 64, 128)),
    }


CALLS = list(operands("cpu"))
NAMES = [(c, n) for c in CALLS for n in operands("cpu")[c]]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="on the GPU is wanted"):
        call(**operands("cpu")[call])


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", NAMES, ids=lambda x: getattr(x, "__name__", x))
def test_one_host_tensor_is_refused(call, name):
    args = operands("cuda")[call]
    call(**args)
    args[name] = args[name].cpu()
    with pytest.raises(ValueError, match=f"{name}: a tensor on the GPU is wanted"):
        call(**args)
    assert tkg.device_status() == tkg.OK


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS[:2], ids=lambda c: c.__name__)
def test_workspaces(call):
    args = operands("cuda")[call]
    ws = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    call(**args, workspace=ws)
    with pytest.raises(ValueError, match="workspace: a tensor on the GPU is wanted"):
        call(**args, workspace=ws.cpu())
    with pytest.raises(ValueError, match="workspace: a contiguous tensor is wanted"):
        call(**args, workspace=ws[::2])
    assert tkg.device_status() == tkg.OK
