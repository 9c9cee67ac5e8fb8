"""GPU: a workspace tells of the last call on it, whichever operator's that was."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", [("rms", "rms"), ("layer", "layer")])
@pytest.mark.parametrize("D", [5, 64, 1000, 8000])
def test_a_backward_clears_what_an_earlier_call_left(D, kinds):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm
    R, V = 7, 900
    print(D, kinds, flush=True)
    p = lm.LogitsPenalty(V)
    w = torch.ones(D, device="cuda")
    n = lm.BlockNorm(D, post=kinds[0], pre=kinds[1], post_weight=w, pre_weight=w)
    ws = torch.zeros(max(p.workspace_bytes(R), n.workspace_bytes(R)), dtype=torch.uint8, device="cuda")
    m = lambda: torch.randn(R, D, device="cuda")  # noqa: E731
    bad = torch.full((R, 4), V, dtype=torch.int32, device="cuda")
    x = torch.randn(R, V, device="cuda")
    for _ in range(2):
        p.apply(x, x, tokens=bad, workspace=ws)
        assert p.device_status(ws) == "SGB_ERR_INDEX_OUT_OF_RANGE"
        n.backward(m(), m(), m(), m(), torch.ones(R, 4, device="cuda"), m(), m(), workspace=ws,
                   d_pre_weight=torch.empty(D, device="cuda"))
        assert n.device_status(ws) == "SGB_OK"
