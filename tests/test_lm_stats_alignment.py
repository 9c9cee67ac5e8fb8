"""CPU: stats that a backward would refuse are refused where they are written."""
import pytest
import torch

from test_lm_abi import BAD, _distill, _norm, refused

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")


def shifted(rows, by):
    buf = torch.zeros(4 * rows + 8)
    at = -buf.data_ptr() % 16 // 4 + by
    return buf[at:at + 4 * rows].view(rows, 4)


@pytest.mark.parametrize("by,code", [(0, "SGB_ERR_HIP"), (1, BAD), (2, BAD), (4, "SGB_ERR_HIP")])
def test_forward_and_backward_agree(by, code):
    n, fwd, bwd = _norm()
    refused(code, n.forward, **{**fwd, "stats": shifted(4, by)})
    refused(code, n.backward, **{**bwd, "stats": shifted(4, by)})
    d, c, loss, grad, _ = _distill()
    refused(code, d.forward, **c, **loss, stats=shifted(3, by))
    refused(code, d.backward, **c, **grad, stats=shifted(3, by), grad_loss=None)
