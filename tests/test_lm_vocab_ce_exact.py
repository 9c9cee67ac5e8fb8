"""CPU: workspaces and refusals of vocabulary cross-entropy with exact gradients."""
import random

import pytest
import torch

from sparse_gradient_backward_amd import lm
from test_lm_step_abi import BAD, HIP, _head, aligned, refused

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_workspaces(dt):
    rng = random.Random(3)
    for _ in range(40):
        D, V = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 23))
        p = lm.VocabCrossEntropy(D, V)
        rows = sorted({int(2 ** rng.uniform(0, 30.9)) for _ in range(12)} | {0, 1, 64, 65, 128, 129, 8192})
        sizes = [p.workspace_bytes(r, dt, exact=True) for r in rows]
        assert sizes == sorted(sizes), (D, V)
        for r, n in zip(rows, sizes):
            assert n >= p.workspace_bytes(r, dt)
            if dt is torch.float32 or r <= 128:
                assert n == p.workspace_bytes(r, dt)
            assert p.workspace_bytes(r, dt, gradient=False, exact=True) == p.workspace_bytes(r, dt, False)


def test_it_stays_bounded():
    for dt in (torch.bfloat16, torch.float16):
        p = lm.VocabCrossEntropy(4096, 131072)
        a, b = (p.workspace_bytes(r, dt, exact=True) for r in (1 << 15, 1 << 20))
        assert b - a <= 8 * (1 << 20) + 1024 and a < 8 << 30


def test_refusals():
    p, c, out, grads = _head(rows=200)
    small = c["workspace"]
    room = aligned(p.workspace_bytes(200, exact=True))
    for kw in (dict(exact=True), dict(exact=True, accumulate=True)):
        refused("SGB_ERR_WORKSPACE_TOO_SMALL", p.loss_grad, **{**c, **out, **grads, "workspace": small}, **kw)
        refused(HIP, p.loss_grad, **{**c, **out, **grads, "workspace": room}, **kw)
        refused(HIP, p.backward, **{**c, **grads, "workspace": room}, lse=out["lse"], **kw)
    refused(HIP, p.loss_grad, **{**c, **out, **grads, "workspace": room})
    # other values of the C call's field
    h, w, dw = 1 << 44, 1 << 45, 1 << 46
    for bits, status in ((-1, BAD), (4, BAD), (0, HIP), (1, HIP), (2, HIP), (3, HIP)):
        args = lm._VOCAB_CE.pack(h, w, 1 << 43, 0, 1 << 42, 0, 0, 0, dw, 24, 24, 0, 24, 200, 1, 1, bits, 1.0)
        code = lm._lib.sgb_vocab_ce_loss_grad(p.handle, args, room.data_ptr(), room.numel() * 8, None)
        assert lm.sgb_status_string(code) == status, bits
    n = lm._sz()
    for gradient in (-1, 3):
        assert lm._lib.sgb_vocab_ce_workspace_bytes(p.handle, 5, 1, gradient, lm.ctypes.byref(n)) == \
            lm.SGB_ERR_INVALID_ARGUMENT
