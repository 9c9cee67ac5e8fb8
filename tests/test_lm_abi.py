"""CPU checks of libsgb_lm.so: its exports, the packed argument structs
against the header's layout, and the refusal of bad arguments.  A plan made
without a GPU checks its calls' arguments and ends valid calls with
SGB_ERR_HIP, so everything the host refuses is tested here."""
import os
import random
import subprocess
import tempfile

import pytest
import torch

import sparse_gradient_backward_amd as sgb
from sparse_gradient_backward_amd import lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")


def test_every_declared_function_is_exported():
    out = subprocess.run(["nm", "-D", "--defined-only", lm.LIB_PATH], capture_output=True,
                         text=True).stdout
    names = lm.header_functions()
    assert len(names) == 16
    for name in names:
        assert f" T {name}\n" in out, name


def test_packed_structs_match_the_header():
    structs = {"sgb_norm_params": lm._NORM_PARAMS, "sgb_norm_forward_args": lm._NORM_FORWARD,
               "sgb_norm_backward_args": lm._NORM_BACKWARD, "sgb_distill_args": lm._DISTILL,
               "sgb_penalty_args": lm._PENALTY}
    # where the first 64-bit integer and the last member start
    last = {"sgb_norm_params": ("post_weight", "dtype", 0, 32),
            "sgb_norm_forward_args": ("x_stride", "res_dtype", 48, 108),
            "sgb_norm_backward_args": ("dx_out_stride", "res_dtype", 104, 188),
            "sgb_distill_args": ("logits_stride", "grad_scale", 80, 124),
            "sgb_penalty_args": ("logits_stride", "dtype", 96, 164)}
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "sgb_lm.h"\nint main(void) {\n'
    for n, (a, b, _, _) in last.items():
        src += f'printf("%zu %zu %zu\\n", sizeof({n}), offsetof({n}, {a}), offsetof({n}, {b}));\n'
    src += "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I",
                               os.path.join(ROOT, "include"), c, "-o", exe])
        lines = subprocess.check_output([exe], text=True).split("\n")
    for line, (n, (_, _, a, b)) in zip(lines, last.items()):
        assert [int(x) for x in line.split()] == [structs[n].size, a, b], n


def refused(code, f, *args, **kw):
    with pytest.raises(sgb.SgbError) as e:
        f(*args, **kw)
    assert e.value.name == code, e.value


BAD = "SGB_ERR_INVALID_ARGUMENT"


def test_plans_refuse_bad_sizes():
    for kw in (dict(D=0), dict(D=8193), dict(D=8, post="batch"), dict(D=8, post_eps=-1.0),
               dict(D=8, pre_eps=float("nan"))):
        refused(BAD, lm.BlockNorm, **kw)
    for a in ((0, 4), (10, 0), (10, 1025), (10, 4, 0.0), (10, 4, -1.0), (10, 4, float("inf")),
              (10, 4, 1.0, float("nan")), (10, 4, 1.0, 1.0, float("inf"))):
        refused(BAD, lm.TopkDistill, *a)
    refused("SGB_ERR_UNSUPPORTED", lm.TopkDistill, 2**23 + 1, 4)
    for v in (0, -1, 2**31):
        refused(BAD, lm.LogitsPenalty, v)
    for p in (lm.BlockNorm(8), lm.TopkDistill(8, 2), lm.LogitsPenalty(8)):
        refused(BAD, p.workspace_bytes, -1)


def _norm(rows=4, D=24, rt=torch.float32, dt=torch.bfloat16, G=2, **kw):
    w = torch.ones(D)
    n = lm.BlockNorm(D, post_weight=w, pre_weight=w.clone(), **kw)
    m = lambda t, r=rows: torch.zeros(r, D, dtype=t)  # noqa: E731
    fwd = dict(x=m(rt), h=m(dt), x_out=m(rt), y=m(dt), gate=m(dt, G), rows_per_gate=2,
               stats=torch.zeros(rows, 4))
    bwd = dict(dx_out=m(rt), dy=m(dt), x_out=m(rt), h=m(dt), stats=torch.zeros(rows, 4), dx=m(rt),
               dh=m(dt), gate=m(dt, G), rows_per_gate=2, d_gate=m(dt, G),
               d_post_weight=torch.zeros(D), d_pre_weight=torch.zeros(D),
               workspace=torch.zeros(n.workspace_bytes(rows) // 8 + 64, dtype=torch.float64))
    ws = bwd["workspace"]
    at = -ws.data_ptr() % 256 // 8
    bwd["workspace"] = ws[at:at + n.workspace_bytes(rows) // 8]
    return n, fwd, bwd


@no_gpu
def test_norm_refusals():
    n, fwd, bwd = _norm()
    refused("SGB_ERR_HIP", n.forward, **fwd)       # valid but for the missing device
    refused("SGB_ERR_HIP", n.backward, **bwd)
    shared = torch.zeros(4, 48)
    for kw in (dict(x=fwd["x"].double()), dict(h=torch.zeros(4, 23, dtype=torch.bfloat16)),
               dict(h=fwd["h"].float()), dict(x=fwd["x"].half(), x_out=fwd["x"].half()),
               dict(y=None), dict(x_out=None), dict(gate=fwd["gate"].float()),
               dict(gate=torch.zeros(3, 24, dtype=torch.bfloat16)), dict(rows_per_gate=0),
               dict(x=torch.zeros(24, 4).t()), dict(stats=torch.zeros(4, 3)),
               dict(x=shared[:, :24], x_out=shared[:, 1:25]),
               dict(x_out=fwd["x"][:1].expand(4, 24)),
               dict(x=fwd["x"][:3]), dict(y=fwd["x_out"].view(torch.bfloat16)[:, :24])):
        refused(BAD, n.forward, **{**fwd, **kw})
    refused("SGB_ERR_HIP", n.forward, **{**fwd, "x_out": fwd["x"], "y": fwd["h"]})
    refused("SGB_ERR_HIP", n.forward, **{**fwd, "x": shared[:, :24], "x_out": shared[:, 24:]})
    for kw in (dict(dy=None), dict(dx=None), dict(stats=None), dict(stats=torch.zeros(17)[1:]),
               dict(gate=None), dict(d_post_bias=torch.zeros(24)),
               dict(d_post_weight=torch.zeros(24).double()), dict(workspace=None),
               dict(dx=bwd["x_out"]), dict(dh=bwd["h"][:, :], dy=None),
               dict(workspace=bwd["workspace"][1:]), dict(d_gate=bwd["d_gate"][:1]),
               dict(d_gate=bwd["gate"]), dict(dx=bwd["dh"].float()[:, :23])):
        refused(BAD, n.backward, **{**bwd, **kw})
    refused("SGB_ERR_WORKSPACE_TOO_SMALL", n.backward,
            **{**bwd, "workspace": bwd["workspace"][:-1]})
    for kw in (dict(dx=bwd["dx_out"]), dict(dh=bwd["dy"]), dict(dh=bwd["h"]),
               dict(d_gate=None, d_post_weight=None, d_pre_weight=None)):
        refused("SGB_ERR_HIP", n.backward, **{**bwd, **kw})
    # parameters: one for each norm there is
    for kw in (dict(post="none"), dict(pre="none")):
        refused(BAD, _norm(**kw)[0].forward, **fwd)
    n.post_weight = None
    refused(BAD, n.forward, **fwd)
    n.post_weight = torch.ones(24).double()
    refused(BAD, n.forward, **fwd)
    n.post_weight = torch.ones(24).half()          # of one type
    refused(BAD, n.forward, **fwd)


@no_gpu
def test_neighbours_in_memory_do_not_overlap():
    """A gate of few rows right before the matrix of many that is written."""
    n, fwd, _ = _norm(dt=torch.float32)
    buf = torch.zeros((2 + 4 + 4) * 24)
    gate, out, y = buf[:48].view(2, 24), buf[48:144].view(4, 24), buf[144:].view(4, 24)
    refused("SGB_ERR_HIP", n.forward, **{**fwd, "gate": gate, "x_out": out, "y": y})
    refused(BAD, n.forward, **{**fwd, "gate": buf[24:72].view(2, 24), "x_out": out, "y": y})


@no_gpu
def test_norm_workspace_holds_every_deal():
    """Rows dealt to teams for any way of sharing gates fit the workspace."""
    rng = random.Random(3)
    for _ in range(4000):
        D = rng.choice((1, 8, 64, 65, 300, 512, 1000, 2048, 4096, 4097, 8192))
        rows = max(1, int(2 ** rng.uniform(0, 17)))
        rpg = max(1, rng.choice((1, 2, 3, rows // 2 + 1, rows // 3 + 1, rows - 1, rows, rows + 1,
                                 2**40, int(2 ** rng.uniform(0, 17)))))
        n = lm.BlockNorm(D)
        far = [(i + 1) << 42 for i in range(20)]   # addresses: nothing is read without a device
        par = lm._NORM_PARAMS.pack(far[0], far[1], far[2], far[3], 0)
        args = lm._NORM_BACKWARD.pack(*far[4:17], *[D] * 8, rows, rpg, 1, 0)
        st = lm._lib.sgb_block_norm_backward(n.handle, par, args, far[18], n.workspace_bytes(rows), 0)
        assert st == sgb.SGB_ERR_HIP, (D, rows, rpg, st)


def _distill(rows=3, V=50, K=4, **kw):
    d = lm.TopkDistill(V, K, ce_weight=0.3, **kw)
    ws = torch.zeros(d.workspace_bytes(rows) // 8 + 64, dtype=torch.float64)
    at = -ws.data_ptr() % 256 // 8
    c = dict(logits=torch.zeros(rows, V), ids=torch.zeros(rows, K, dtype=torch.int64),
             values=torch.zeros(rows, K), teacher_lse=torch.zeros(rows),
             labels=torch.zeros(rows, dtype=torch.int64), row_weights=torch.ones(rows),
             workspace=ws[at:at + d.workspace_bytes(rows) // 8])
    return d, c, dict(loss=torch.zeros(rows)), dict(grad=torch.zeros(rows, V)), \
        dict(stats=torch.zeros(rows, 4))


@no_gpu
def test_distill_refusals():
    d, c, loss, grad, stats = _distill()
    refused("SGB_ERR_HIP", d.forward, **c, **loss)
    refused("SGB_ERR_HIP", d.forward, **c, **loss, **stats)
    refused("SGB_ERR_HIP", d.loss_grad, **c, **loss, **grad)
    refused("SGB_ERR_HIP", d.backward, **c, **stats, **grad, grad_loss=None)
    for kw in (dict(logits=c["logits"].double()), dict(logits=torch.zeros(3, 49)),
               dict(ids=c["ids"].int()), dict(values=c["values"].half()), dict(ids=c["ids"][:, :3]),
               dict(labels=None), dict(labels=torch.zeros(3)), dict(teacher_lse=torch.zeros(2)),
               dict(row_weights=torch.ones(6)[::2]), dict(workspace=None), dict(loss=None),
               dict(grad=None), dict(grad=c["logits"]), dict(grad_scale=float("nan")),
               dict(grad=torch.zeros(3, 50).half()), dict(workspace=c["workspace"][1:])):
        refused(BAD, d.loss_grad, **{**c, **loss, **grad, **kw})
    refused(BAD, d.backward, **c, stats=None, grad_loss=None, **grad)
    refused(BAD, d.backward, **c, stats=torch.zeros(13)[1:], grad_loss=None, **grad)
    refused("SGB_ERR_WORKSPACE_TOO_SMALL", d.forward,
            **{**c, **loss, "workspace": c["workspace"][:32]})
    d2 = lm.TopkDistill(50, 4)                     # no cross-entropy: no labels
    refused(BAD, d2.forward, **c, **loss)


@no_gpu
def test_penalty_refusals():
    p = lm.LogitsPenalty(50)
    buf = torch.zeros(128, dtype=torch.float64)
    ws = buf[-buf.data_ptr() % 256 // 8:][:32]
    i32 = torch.int32
    c = dict(logits=torch.zeros(3, 50), out=torch.zeros(3, 50),
             tokens=torch.zeros(3, 6, dtype=i32), prompt_lens=torch.zeros(3, dtype=i32),
             lens=torch.zeros(3, dtype=i32), repetition=torch.ones(3), frequency=torch.ones(3),
             presence=torch.ones(3), bias_ids=torch.zeros(3, 2, dtype=i32),
             bias_values=torch.zeros(3, 2), mask=torch.zeros(2, 2, dtype=i32),
             mask_index=torch.zeros(3, dtype=i32), workspace=ws)
    refused("SGB_ERR_HIP", p.apply, **c)
    refused("SGB_ERR_HIP", p.apply, **{**c, "out": c["logits"]})
    wide = torch.zeros(3, 120)
    for kw in (dict(logits=torch.zeros(3, 51)), dict(out=torch.zeros(3, 50).half()), dict(out=None),
               dict(tokens=c["tokens"].long()), dict(lens=torch.zeros(3)),
               dict(repetition=torch.ones(4)), dict(bias_values=None),
               dict(bias_values=torch.zeros(3, 3)), dict(mask=torch.zeros(2, 1, dtype=i32)),
               dict(mask_index=None), dict(workspace=None), dict(tokens=c["tokens"][:2]),
               dict(logits=wide[:, :50], out=wide[:, 20:70])):
        refused(BAD, p.apply, **{**c, **kw})
    refused("SGB_ERR_HIP", p.apply, **{**c, "logits": wide[:, :50], "out": wide[:, 60:110]})
    refused("SGB_ERR_WORKSPACE_TOO_SMALL", p.apply, **{**c, "workspace": ws[:31]})
    refused("SGB_ERR_UNSUPPORTED", p.apply, **{**c, "bias_ids": torch.zeros(3, 1024, dtype=i32),
                                               "bias_values": torch.zeros(3, 1024)})
    refused("SGB_ERR_UNSUPPORTED", p.apply, **{**c, "tokens": torch.zeros(3, 2**21, dtype=i32)})


def test_null_arguments():
    lib = lm._lib
    assert lib.sgb_block_norm_forward(None, None, None, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    assert lib.sgb_block_norm_backward(None, None, None, None, 0, None) == \
        sgb.SGB_ERR_INVALID_ARGUMENT
    for f in (lib.sgb_distill_forward, lib.sgb_distill_backward, lib.sgb_distill_loss_grad,
              lib.sgb_penalty_apply):
        assert f(None, None, None, 0, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    assert lib.sgb_lm_device_status(None, None, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    for k in ("block_norm", "distill", "penalty"):
        getattr(lib, f"sgb_{k}_destroy")(None)
