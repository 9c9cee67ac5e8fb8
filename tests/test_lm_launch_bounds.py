"""CPU: calls of more rows than one launch takes are refused by name before
anything is enqueued; those just below are not."""
import pytest
import torch

import sparse_gradient_backward_amd as sgb
from sparse_gradient_backward_amd import lm

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")
FAR = [(i + 1) << 42 for i in range(14)]      # addresses: nothing is read without a device
UNSUPPORTED, HIP = 2, 6


def distill(V, rows, call, dtype=0):
    d = lm.TopkDistill(V, 4)
    args = lm._DISTILL.pack(*FAR[:4], 0, *FAR[5:8], 0, FAR[9], V, 4, 4, V, rows, dtype, 1.0)
    return getattr(lm._lib, f"sgb_distill_{call}")(d.handle, args, FAR[10],
                                                   d.workspace_bytes(rows), 0)


@pytest.mark.parametrize("call", ["forward", "backward", "loss_grad"])
@pytest.mark.parametrize("V,most", [(8, 2**24 - 1), (8192, 2**24 - 1)])
def test_distill(V, most, call):
    assert sgb.SGB_ERR_HIP == HIP
    assert distill(V, most, call) == HIP
    for rows in (most + 1, 2**25 - 1):
        assert distill(V, rows, call) == UNSUPPORTED


def test_distill_of_longer_rows():
    for V, most in ((8193, 2**23 - 1), (32769, 2**22 - 1)):
        for call in ("forward", "loss_grad"):
            assert distill(V, most, call) == HIP
            assert distill(V, most + 1, call) == UNSUPPORTED
    # rows that several workgroups share
    assert distill(2**23, 2**18 - 1, "loss_grad") == HIP
    assert distill(2**23, 2**18, "loss_grad") == UNSUPPORTED


@pytest.mark.parametrize("V,L,most", [(50, 0, 2**23 - 1), (50, 20000, 2**22 - 1),
                                      (131072, 0, 2**19 - 1)])
def test_penalties(V, L, most):
    p = lm.LogitsPenalty(V)

    def status(rows):
        args = lm._PENALTY.pack(FAR[0], FAR[1], FAR[2], *[0] * 9, V, V, L, 0, 0, 0, rows, L, 0, 0, 0)
        return lm._lib.sgb_penalty_apply(p.handle, args, FAR[3], 256, 0)
    assert status(most) == HIP
    assert status(most + 1) == UNSUPPORTED
