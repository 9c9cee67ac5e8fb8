"""CPU: a workspace made for some rows serves any fewer."""
import pytest
import torch

from sparse_gradient_backward_amd import lm
import sparse_gradient_backward_amd as sgb

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")


@pytest.mark.parametrize("V", [1, 8, 2048, 2049, 16384, 50021, 131072, 131073, 151936, 2**23])
def test_distill_workspace_grows_with_the_rows(V):
    d = lm.TopkDistill(V, 4)
    sizes = [d.workspace_bytes(r) for r in list(range(0, 2500)) + [2**k for k in range(12, 25)]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("make", [lambda: lm.BlockNorm(24), lambda: lm.BlockNorm(4096),
                                  lambda: lm.BlockNorm(8192), lambda: lm.LogitsPenalty(50021)])
def test_the_others_do_too(make):
    p = make()
    sizes = [p.workspace_bytes(r) for r in list(range(0, 2500)) + [2**k for k in range(12, 31)]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@no_gpu
@pytest.mark.parametrize("V", [100, 50021, 131072, 140001])
def test_every_row_count_takes_a_workspace_for_more(V):
    """Not refused for its size: a plan without a device ends valid calls in SGB_ERR_HIP."""
    d = lm.TopkDistill(V, 4)
    far = [(i + 1) << 42 for i in range(12)]     # addresses: nothing is read without a device
    for most in (40, 512, 1024, 2000):
        n = d.workspace_bytes(most)
        for rows in range(1, most + 1):
            args = lm._DISTILL.pack(*far[:4], 0, *far[5:8], 0, far[9], V, 4, 4, V, rows, 0, 1.0)
            for call in ("forward", "backward", "loss_grad"):
                st = getattr(lm._lib, f"sgb_distill_{call}")(d.handle, args, far[10], n, 0)
                assert st == sgb.SGB_ERR_HIP, (V, most, rows, call, st)
