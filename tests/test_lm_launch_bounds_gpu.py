"""GPU: as many rows as one launch takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_the_most_rows_of_a_distillation():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm, SgbError
    rows, V = 2**24 - 1, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(rows + 1, V, generator=g, device="cuda")
    ids = torch.randint(0, V, (rows + 1, 1), generator=g, device="cuda")
    vals = torch.zeros(rows + 1, 1, device="cuda")
    loss, grad = torch.empty(rows + 1, device="cuda"), torch.empty_like(x)
    d = lm.TopkDistill(V, 1)
    ws = d.workspace(rows + 1)
    with pytest.raises(SgbError) as e:
        d.loss_grad(x, ids, vals, loss, grad, workspace=ws)
    assert e.value.name == "SGB_ERR_UNSUPPORTED"
    d.loss_grad(x[:rows], ids[:rows], vals[:rows], loss[:rows], grad[:rows], workspace=ws)
    # one listed id: the cross-entropy at it.  fp32 roundings on either side: 64 of
    # values below 16
    lq = torch.log_softmax(x[:rows], 1)
    assert float((loss[:rows] + lq.gather(1, ids[:rows])[:, 0]).abs().max()) < 64 * 2.0**-24 * 16
    want = lq.exp_().scatter_add_(1, ids[:rows], torch.full_like(vals[:rows], -1.0))
    assert float((grad[:rows] - want).abs().max()) < 64 * 2.0**-24
