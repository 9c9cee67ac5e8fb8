"""GPU: a short last batch on the workspace of a full one."""
import pytest
import torch

import lm_strict as strict
import test_lm_distill_gpu as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,rows,V", [(1024, 1000, 9001), (64, 37, 20011), (512, 130, 17001)])
def test_fewer_rows_on_a_larger_workspace(most, rows, V):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm
    print(most, rows, V, flush=True)
    c = base.make(rows, V, 8, "bf16", 1.0, True, 0.3)
    d = lm.TopkDistill(V, 8, kd_weight=0.7, ce_weight=0.3)
    cu = {k: v.cuda() for k, v in c.items()}
    loss, grad = torch.empty(rows, device="cuda"), torch.empty_like(cu["x"])
    ws = d.workspace(most)
    kw = dict(teacher_lse=cu["lse"], labels=cu["labels"], row_weights=cu["w"], workspace=ws)
    d.loss_grad(cu["x"], cu["ids"], cu["vals"], loss, grad, **kw)
    stats, loss2, grad2 = torch.empty(rows, 4, device="cuda"), torch.empty_like(loss), torch.empty_like(grad)
    d.forward(cu["x"], cu["ids"], cu["vals"], loss2, stats=stats, **kw)
    d.backward(cu["x"], cu["ids"], cu["vals"], stats, None, grad2, **kw)
    want = base.ref.distill(c["x"], c["ids"], c["vals"], 1.0, 0.7, 0.3, c["lse"], c["labels"], c["w"])
    strict.check(dict(loss=loss, grad=grad), want, "loss_grad")
    strict.check(dict(loss=loss2, grad=grad2), want, "forward, backward")
