"""CPU: a gradient scale that no C float holds is refused like any other argument."""
import pytest
import torch

from test_lm_abi import _distill
from test_lm_step_abi import BAD, HIP, _head, refused

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")
SCALES = (1e39, -1e39, 3.4028236e38, float("inf"), float("nan"))


@no_gpu
@pytest.mark.parametrize("scale", SCALES)
def test_head(scale):
    p, c, out, grads = _head()
    refused(BAD, p.loss_grad, **c, **out, **grads, grad_scale=scale)
    refused(BAD, p.backward, **c, lse=out["lse"], **grads, grad_scale=scale)
    refused(HIP, p.loss_grad, **c, **out, **grads, grad_scale=3.4028234e38)


@no_gpu
@pytest.mark.parametrize("scale", SCALES)
def test_distillation(scale):
    p, c, loss, grad, _ = _distill()
    refused(BAD, p.loss_grad, **c, **loss, **grad, grad_scale=scale)
    refused(HIP, p.loss_grad, **c, **loss, **grad, grad_scale=-3.4028234e38)
