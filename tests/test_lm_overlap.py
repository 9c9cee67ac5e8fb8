"""CPU: block norms' backward refuses outputs that lie over each other or over
what is still read, and takes neighbours that do not."""
import pytest
import torch

from test_lm_abi import BAD, _norm, refused

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")
OK = "SGB_ERR_HIP"      # a valid call, but for the missing device


def call(code, **kw):
    n, _, bwd = _norm(dt=torch.float32)
    refused(code, n.backward, **{**bwd, **kw})


def test_d_gate():
    n, _, bwd = _norm(dt=torch.float32)
    for k in ("dx_out", "dy", "x_out", "h", "dx", "dh"):
        refused(BAD, n.backward, **{**bwd, "d_gate": bwd[k][1:3]})
    refused(OK, n.backward, **bwd)
    # a gate's gradient beside the rows of a wider buffer, and among them
    wide = torch.zeros(4, 60)
    call(OK, dx=wide[:, :24], d_gate=wide[:2, 24:48])
    call(BAD, dx=wide[:, :24], d_gate=wide[:2, 23:47])


def test_the_parameters_gradients():
    n, _, bwd = _norm(dt=torch.float32)
    for k in ("dx", "dh", "d_gate"):
        refused(BAD, n.backward, **{**bwd, "d_pre_weight": bwd[k][1]})
    both = torch.zeros(48)
    call(BAD, d_post_weight=both[:24], d_pre_weight=both[23:47])
    call(OK, d_post_weight=both[:24], d_pre_weight=both[24:])
    # a vector between the rows of a wider buffer, and one that reaches into them
    wide = torch.zeros(4, 60)
    call(OK, dx=wide[:, :24], d_pre_weight=wide[2, 24:48])
    call(OK, dx=wide[:, 36:], d_pre_weight=wide[2, 12:36])
    call(BAD, dx=wide[:, :24], d_pre_weight=wide[2, 20:44])
    call(BAD, dx=wide[:, 36:], d_pre_weight=wide[2, 13:37])
    # one flat buffer of gradients
    flat = torch.zeros(4 * 24)
    call(OK, d_gate=flat[:48].view(2, 24), d_post_weight=flat[48:72], d_pre_weight=flat[72:])


def test_a_single_row_between_others():
    """One gate row in the gap of the rows that are written (forward)."""
    n, fwd, _ = _norm(dt=torch.float32)
    wide = torch.zeros(4, 60)
    args = {**fwd, "rows_per_gate": 4, "x_out": wide[:, :24]}
    for at, code in ((24, OK), (36, OK), (20, BAD), (37, BAD)):
        gate = wide.view(-1)[60 + at:60 + at + 24].view(1, 24)
        refused(code, n.forward, **{**args, "gate": gate})
