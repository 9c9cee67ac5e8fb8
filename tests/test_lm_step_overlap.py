"""CPU: the step's operators refuse every output that lies over something else of
the call, vectors and workspaces too, and take neighbours that do not."""
import pytest
import torch

from sparse_gradient_backward_amd import lm
from test_lm_step_abi import BAD, HIP, _head, aligned, i64, refused

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")


def as_type(t, dtype):
    """The bytes of t as a vector of another type."""
    return t.reshape(-1).view(torch.uint8).view(dtype)


def test_quantising_norm():
    n = lm.QuantNorm(72, weight=torch.ones(72), group=32)
    c = dict(h=torch.zeros(4, 72), x=torch.zeros(4, 72), x_out=torch.zeros(4, 72),
             q=torch.zeros(4, 72, dtype=torch.int8), scales=torch.zeros(4, 3), stats=torch.zeros(4, 4))
    refused(HIP, n.forward, **c)
    for k in ("h", "x", "x_out"):
        refused(BAD, n.forward, **{**c, "scales": c[k][:, :3]})
        refused(BAD, n.forward, **{**c, "scales": c[k][:, 69:]})
        refused(BAD, n.forward, **{**c, "stats": as_type(c[k], torch.float32)[48:64].view(4, 4)})
    q = as_type(c["q"], torch.float32)                   # 72 floats
    refused(BAD, n.forward, **{**c, "scales": q[60:].view(4, 3)})
    refused(BAD, n.forward, **{**c, "stats": q[56:].view(4, 4)})
    refused(BAD, n.forward, **{**c, "scales": c["stats"][:, :3]})
    w = torch.ones(72)
    n.weight = w
    refused(HIP, n.forward, **c)
    for k, over in (("x_out", w.view(1, 72)), ("scales", w[60:63].view(1, 3)), ("stats", w[68:].view(1, 4)),
                    ("q", as_type(w, torch.int8)[200:272].view(1, 72))):
        one = {name: t[:1] for name, t in c.items()}
        refused(HIP, n.forward, **one)
        refused(BAD, n.forward, **{**one, k: over})
    n.weight = torch.ones(72)
    # codes and scales side by side in rows of one buffer of bytes
    rows = torch.zeros(4, 88, dtype=torch.uint8)
    beside = dict(q=rows[:, :72].view(torch.int8), scales=rows.view(torch.float32)[:, 18:21])
    refused(HIP, n.forward, **{**c, **beside})
    refused(BAD, n.forward, **{**c, **beside, "scales": rows.view(torch.float32)[:, 17:20]})
    # in place, and still nothing else on it
    refused(HIP, n.forward, **{**c, "x_out": c["x"]})
    refused(BAD, n.forward, **{**c, "x_out": c["x"], "scales": c["x"][:, :3]})


def test_dropout_state():
    d = lm.Dropout(0.1)
    x, out = torch.zeros(4, 24), torch.zeros(4, 24)
    refused(HIP, d.forward, x, out, state=torch.zeros(2, dtype=i64))
    refused(BAD, d.forward, x, out, state=as_type(out, i64)[:2])
    refused(BAD, d.forward, x, out, state=as_type(out, i64)[46:])
    wide = torch.zeros(4, 28)
    refused(HIP, d.forward, x, wide[:, :24], state=as_type(wide, i64)[12:14])


def test_head():
    p, c, out, grads = _head(dt=torch.float32)           # 3 rows of 24, 50 tokens
    every = {**c, **out, **grads}
    refused(HIP, p.loss_grad, **every)
    refused(BAD, p.loss_grad, **{**every, "lse": out["loss"]})
    for k in ("hidden", "weight", "d_hidden", "d_weight"):
        for o in ("loss", "lse"):
            refused(BAD, p.loss_grad, **{**every, o: every[k].view(-1)[30:33]})
    for o in ("loss", "lse"):
        refused(BAD, p.loss_grad, **{**every, o: c["row_weights"]})
        refused(BAD, p.loss_grad, **{**every, o: as_type(c["labels"], torch.float32)[3:]})
        refused(BAD, p.forward, **{**c, **out, o: c["row_weights"]})
    lots = torch.zeros(10, 24)
    lab = lots.view(-1).view(torch.uint8).view(i64)[3:6]
    refused(BAD, p.loss_grad, **{**every, "d_hidden": lots[:3], "labels": lab})
    # a backward reads lse and the gradients from above
    back = {**c, **grads, "lse": out["lse"], "grad_loss": torch.ones(3)}
    refused(HIP, p.backward, **back)
    refused(HIP, p.backward, **{**back, "grad_loss": out["lse"]})
    for k in ("lse", "grad_loss"):
        for o in ("d_hidden", "d_weight"):
            refused(BAD, p.backward, **{**back, k: grads[o].view(-1)[-3:]})
    # the workspace
    ws = aligned(p.workspace_bytes(3, torch.float32) + 8192)
    head = torch.as_tensor(ws).view(torch.float32)
    assert ws.data_ptr() % 256 == 0
    for k, t in (("hidden", head[:72].view(3, 24)), ("weight", head[64:1264].view(50, 24)),
                 ("loss", head[100:103]), ("lse", head[:3]), ("d_hidden", head[8:80].view(3, 24)),
                 ("d_weight", head[:1200].view(50, 24)), ("labels", ws.view(i64)[:3]),
                 ("row_weights", head[5:8])):
        refused(BAD, p.loss_grad, **{**every, "workspace": ws, k: t})
    n = p.workspace_bytes(3, torch.float32) // 4         # behind what the call uses
    refused(HIP, p.loss_grad, **{**every, "workspace": ws, "loss": head[n:n + 3]})
    # a vector in the gap of a wider buffer's rows
    wide = torch.zeros(3, 40)
    refused(HIP, p.loss_grad, **{**every, "d_hidden": wide[:, :24], "loss": wide[1, 24:27]})
    refused(BAD, p.loss_grad, **{**every, "d_hidden": wide[:, :24], "loss": wide[1, 23:26]})
