"""CPU checks of sgb_lm_step.h's operators: exports, the packed argument structs
against the header's layout, refusals, workspaces.  A plan made without a GPU
checks its calls' arguments and ends valid calls with SGB_ERR_HIP."""
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
BAD, HIP, UNSUPPORTED = "SGB_ERR_INVALID_ARGUMENT", "SGB_ERR_HIP", "SGB_ERR_UNSUPPORTED"
f32, bf16, f16, i64 = torch.float32, torch.bfloat16, torch.float16, torch.int64


def refused(status, f, *a, **kw):
    with pytest.raises(sgb.SgbError) as e:
        f(*a, **kw)
    assert status in str(e.value), str(e.value)


def test_every_declared_function_is_exported():
    out = subprocess.run(["nm", "-D", "--defined-only", lm.LIB_PATH], capture_output=True,
                         text=True).stdout
    names = lm.header_functions(lm.STEP_HEADER)
    assert len(names) == 12
    for name in names:
        assert f" T {name}\n" in out, name


def test_packed_structs_match_the_header():
    structs = {"sgb_vocab_ce_args": lm._VOCAB_CE, "sgb_dropout_args": lm._DROPOUT,
               "sgb_quant_norm_args": lm._QUANT_NORM}
    # where the first 64-bit integer and the last member start
    last = {"sgb_vocab_ce_args": ("hidden_stride", "grad_scale", 72, 124),
            "sgb_dropout_args": ("x_stride", "reserved", 32, 100),
            "sgb_quant_norm_args": ("h_stride", "reserved", 56, 116)}
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "sgb_lm_step.h"\nint main(void) {\n'
    for n, (a, b, _, _) in last.items():
        src += f'printf("%zu %zu %zu\\n", sizeof({n}), offsetof({n}, {a}), offsetof({n}, {b}));\n'
    src += "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                        c, "-o", exe], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (n, (_, _, x, y)) in zip(got, last.items()):
        assert line == f"{structs[n].size} {x} {y}", n


def test_plans_refuse_bad_sizes():
    for a in ((0, 5), (-1, 5), (5, 0), (5, -1)):
        refused(BAD, lm.VocabCrossEntropy, *a)
    for a in ((16385, 5), (5, 2**23 + 1)):
        refused(UNSUPPORTED, lm.VocabCrossEntropy, *a)
    refused(BAD, lm.VocabCrossEntropy, 2**32 + 8, 5)
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        refused(BAD, lm.Dropout, p)
    for kw in (dict(D=0), dict(D=8193), dict(D=2**32 + 8), dict(D=8, group=16), dict(D=8, group=1024),
               dict(D=8, group=-32), dict(D=8, form="int4"), dict(D=8, eps=-1.0),
               dict(D=8, eps=float("nan")), dict(D=8, eps=float("inf"))):
        refused(BAD, lm.QuantNorm, **kw)
    p = lm.VocabCrossEntropy(8, 8)
    for rows in (-1, 2**31):
        refused(BAD, p.workspace_bytes, rows)
    refused(BAD, p.workspace_bytes, 4, torch.float64)


def aligned(n):
    """n bytes (a multiple of 8) at an address of 256."""
    buf = torch.zeros(n // 8 + 64, dtype=torch.float64)
    return buf[-buf.data_ptr() % 256 // 8:][:n // 8]


def _head(rows=3, D=24, V=50, dt=bf16, wt=None):
    p = lm.VocabCrossEntropy(D, V)
    c = dict(hidden=torch.zeros(rows, D, dtype=dt), weight=torch.zeros(V, D, dtype=dt),
             labels=torch.zeros(rows, dtype=i64), row_weights=torch.ones(rows),
             workspace=aligned(p.workspace_bytes(rows, dt)))
    return p, c, dict(loss=torch.zeros(rows), lse=torch.zeros(rows)), \
        dict(d_hidden=torch.zeros(rows, D, dtype=dt), d_weight=torch.zeros(V, D, dtype=wt or dt))


@no_gpu
def test_head_refusals():
    p, c, out, grads = _head()
    lse = dict(lse=out["lse"])
    refused(HIP, p.forward, **c, **out)
    refused(HIP, p.loss_grad, **c, **out, **grads)
    refused(HIP, p.loss_grad, **c, loss=out["loss"])          # nothing but the loss wanted
    refused(HIP, p.loss_grad, **c, **out, d_hidden=grads["d_hidden"])
    refused(HIP, p.loss_grad, **c, **out, d_weight=torch.zeros(50, 24))
    refused(HIP, p.backward, **c, **lse, **grads, grad_loss=torch.ones(3))
    wide = torch.zeros(3, 100, dtype=bf16)
    rows = torch.zeros(53, 24, dtype=bf16)
    for kw in (dict(hidden=c["hidden"].double()), dict(hidden=c["hidden"][:, :23]),
               dict(hidden=torch.zeros(24, 3, dtype=bf16).t()), dict(weight=c["weight"].float()),
               dict(weight=c["weight"][:49]), dict(labels=c["labels"].int()),
               dict(labels=c["labels"][:2]), dict(labels=None), dict(row_weights=torch.ones(6)[::2]),
               dict(loss=None), dict(loss=torch.zeros(3).double()), dict(lse=torch.zeros(4)),
               dict(d_hidden=torch.zeros(3, 24)), dict(d_weight=torch.zeros(50, 24, dtype=f16)),
               dict(d_weight=torch.zeros(49, 24, dtype=bf16)), dict(grad_scale=float("nan")),
               dict(workspace=None), dict(workspace=c["workspace"][1:]),
               dict(d_hidden=c["hidden"]), dict(d_weight=c["weight"]),
               dict(d_weight=rows[:50], d_hidden=rows[49:52]),
               dict(hidden=wide[:, :24], d_hidden=wide[:, 20:44]),
               dict(hidden=rows[:3], d_weight=rows[2:52]),
               dict(weight=c["weight"][:1].expand(50, 24), d_weight=c["weight"])):
        refused(BAD, p.loss_grad, **{**c, **out, **grads, **kw})
    refused(HIP, p.loss_grad, **{**c, **out, **grads, "hidden": wide[:, :24], "d_hidden": wide[:, 24:48]})
    refused("SGB_ERR_WORKSPACE_TOO_SMALL", p.loss_grad,
            **{**c, **out, **grads, "workspace": c["workspace"][:-1]})
    small = aligned(p.workspace_bytes(3, bf16, gradient=False))
    refused(HIP, p.forward, **{**c, "workspace": small}, **out)
    refused("SGB_ERR_WORKSPACE_TOO_SMALL", p.loss_grad, **{**c, "workspace": small}, **out, **grads)
    refused(BAD, p.backward, **c, lse=None, **grads)
    refused(BAD, p.backward, **c, **lse)                       # no gradient wanted
    refused(BAD, p.backward, **c, **lse, **grads, grad_loss=torch.ones(2))


@no_gpu
@pytest.mark.parametrize("dt", [f32, bf16, f16])
def test_head_workspaces_serve_fewer_rows(dt):
    rng = random.Random(2)
    for _ in range(40):
        D, V = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 23))
        p = lm.VocabCrossEntropy(D, V)
        for gradient in (False, True):
            rows = sorted({int(2 ** rng.uniform(0, 30.9)) for _ in range(12)} | {0, 1, 2, 63, 64, 65, 8192})
            sizes = [p.workspace_bytes(r, dt, gradient) for r in rows]
            assert sizes == sorted(sizes), (D, V, gradient)
        assert p.workspace_bytes(100, dt, False) <= p.workspace_bytes(100, dt, True)


@no_gpu
def test_head_workspace_does_not_grow_past_a_chunk():
    """But for the rows' own log-sum-exps and label logits."""
    for dt in (f32, bf16, f16):
        p = lm.VocabCrossEntropy(4096, 131072)
        a, b = (p.workspace_bytes(r, dt) for r in (1 << 15, 1 << 20))
        assert b - a <= 8 * (1 << 20) + 1024
        assert a < 7 << 30


@no_gpu
def test_dropout_refusals():
    d = lm.Dropout(0.1)
    x, out = torch.zeros(4, 24), torch.zeros(4, 24)
    refused(HIP, d.forward, x, out, 1, 2)
    refused(HIP, d.forward, x, x, 1, 2)
    refused(HIP, d.forward, x, out, 2**64 - 1, 2**64 - 1, residual=torch.zeros(4, 24), first_row=2**62 - 4)
    refused(HIP, d.forward, x, out, residual=out)
    refused(HIP, d.forward, x.half(), out, residual=torch.zeros(4, 24))
    refused(HIP, d.backward, x, out, 1)
    wide = torch.zeros(4, 60)
    refused(HIP, d.forward, wide[:, :24], wide[:, 24:48], 1)
    for a, kw in (((x.double(), out), {}), ((x, out.half()), {}), ((x.half(), out), {}),
                  ((x, out[:3]), {}), ((x, torch.zeros(4, 23)), {}), ((x, None), {}),
                  ((x, torch.zeros(24, 4).t()), {}), ((x[0], out[0]), {}),
                  ((x, out, -1), {}), ((x, out, 2**64), {}), ((x, out, 1, -1), {}),
                  ((x, out), dict(residual=torch.zeros(4, 24).half())),
                  ((x, out), dict(residual=torch.zeros(4, 25))),
                  ((x.half(), out.bfloat16()), dict(residual=out.bfloat16())),
                  ((x, out), dict(first_row=-1)), ((x, out), dict(first_row=2**62 - 3)),
                  ((x, out), dict(state=torch.zeros(2))), ((x, out), dict(state=torch.zeros(3, dtype=i64))),
                  ((wide[:, :24], wide[:, 20:44]), {}),
                  ((x.half(), out), dict(residual=x.half())),
                  ((x, torch.zeros(1, 24).expand(4, 24)), {})):
        refused(BAD, d.forward, *a, **kw)
    refused(BAD, d.forward, torch.zeros(4, 0), torch.zeros(4, 0))
    refused(UNSUPPORTED, d.forward, torch.zeros(1, 2**24 + 1, dtype=f16), torch.zeros(1, 2**24 + 1, dtype=f16))
    # more rows than one launch takes: those just below are not refused
    far = [(i + 1) << 44 for i in range(4)]
    for cols, most in ((1, 2**34 - 2**10), (2048, (2**24 - 1) * 4)):
        for rows, status in ((most, sgb.SGB_ERR_HIP), (most + 2**10, 2)):
            args = lm._DROPOUT.pack(far[0], 0, far[2], 0, cols, 0, cols, rows, 0, 1, 0, cols, 0, 0, 0)
            assert lm._lib.sgb_dropout_apply(d.handle, args, 0) == status, (cols, rows)


@no_gpu
def test_quant_refusals():
    n = lm.QuantNorm(72, weight=torch.ones(72), group=32)
    c = dict(h=torch.zeros(4, 72, dtype=bf16), x=torch.zeros(4, 72), x_out=torch.zeros(4, 72),
             q=torch.zeros(4, 72, dtype=torch.int8), scales=torch.zeros(4, 3), stats=torch.zeros(4, 4))
    refused(HIP, n.forward, **c)
    for kw in (dict(x=None, x_out=None), dict(x=None), dict(x_out=None), dict(stats=None),
               dict(x_out=c["x"]), dict(x=c["h"].clone(), x_out=c["h"])):
        refused(HIP, n.forward, **{**c, **kw})
    wide = torch.zeros(4, 200)
    refused(HIP, n.forward, **{**c, "x": wide[:, :72], "x_out": wide[:, 72:144]})
    for kw in (dict(h=c["h"].double()), dict(h=c["h"][:, :71]), dict(x=c["x"].half()),
               dict(x=c["x"].double(), x_out=None), dict(x_out=c["h"]), dict(q=None),
               dict(q=torch.zeros(4, 72, dtype=torch.uint8)), dict(q=c["q"][:3]), dict(scales=None),
               dict(scales=torch.zeros(4, 2)), dict(scales=torch.zeros(4, 3).double()),
               dict(stats=torch.zeros(3, 4)), dict(stats=torch.zeros(17)[1:].view(4, 4)),
               dict(x=wide[:, :72], x_out=wide[:, 70:142]),
               dict(q=c["h"].view(torch.int8)[:, :72]),
               dict(q=torch.zeros(1, 72, dtype=torch.int8).expand(4, 72))):
        refused(BAD, n.forward, **{**c, **kw})
    for w in (None, torch.ones(71), torch.ones(72).double(), torch.ones(144)[::2]):
        n.weight = w
        refused(BAD, n.forward, **c)


def test_null_arguments():
    lib = lm._lib
    for f in (lib.sgb_vocab_ce_forward, lib.sgb_vocab_ce_backward, lib.sgb_vocab_ce_loss_grad):
        assert f(None, None, None, 0, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    assert lib.sgb_dropout_apply(None, None, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    assert lib.sgb_quant_norm_forward(None, None, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    assert lib.sgb_vocab_ce_workspace_bytes(None, 1, 0, 0, None) == sgb.SGB_ERR_INVALID_ARGUMENT
    for k in ("vocab_ce", "dropout", "quant_norm"):
        getattr(lib, f"sgb_{k}_destroy")(None)
        assert getattr(lib, f"sgb_{k}_create")(None, *{"vocab_ce": (8, 8), "dropout": (0.5,),
                                                       "quant_norm": (8, 0, 0, 0.0)}[k]) == \
            sgb.SGB_ERR_INVALID_ARGUMENT
