"""Python binding of libsgb_lm.so, the token-model operators (C ABI:
``include/sgb_lm.h`` and ``include/sgb_lm_step.h``): block norms, distillation
from a teacher's top logits, logits penalties; vocabulary cross-entropy,
dropout, quantising norms.

Argument marshalling only: the computation runs in the library's HIP kernels.
Every tensor is a device tensor on the plan's GPU; matrices are 2-D with
adjacent elements in a row and any row stride, vectors are contiguous.
`stream` is a torch stream (default: the current one); work is enqueued there
and the call returns at once, so tensors last used on another stream need the
caller's ordering, as with any kernel.  Errors are ``SgbError``.  Importing
this module fails loudly (ImportError) when the library has not been built.

    norm = lm.BlockNorm(4096, post="rms", pre="rms", post_weight=w1, pre_weight=w2)
    norm.forward(x, h, x_out, y, gate=gate, rows_per_gate=1024, stats=stats)
    norm.backward(dx_out, dy, x_out, h, stats, dx, dh, gate=gate, rows_per_gate=1024,
                  d_gate=dg, d_post_weight=dw1, d_pre_weight=dw2, workspace=ws)

    head = lm.VocabCrossEntropy(4096, 131072)
    head.loss_grad(y, table, labels, loss, d_y, d_table, grad_scale=1 / tokens,
                   workspace=head.workspace(tokens, torch.bfloat16))
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

import torch

from . import (DTYPE, SGB_ERR_INVALID_ARGUMENT, SgbError, _check, sgb_status_string)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("SGB_LM_LIBRARY") or os.path.join(_HERE, "libsgb_lm.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "sgb_lm.h")
STEP_HEADER = os.path.join(os.path.dirname(_HERE), "include", "sgb_lm_step.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python sparse_gradient_backward_amd/build.py` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)
_vp, _i32, _i64, _f32, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                              ctypes.c_size_t)
_out = ctypes.POINTER(_vp)
for _name, _args in {
        "sgb_lm_device_status": [_vp, _vp, ctypes.POINTER(_i32)],
        "sgb_block_norm_create": [_out, _i32, _i32, _i32, _f32, _f32, _f32],
        "sgb_block_norm_destroy": [_vp],
        "sgb_block_norm_workspace_bytes": [_vp, _i64, ctypes.POINTER(_sz)],
        "sgb_block_norm_forward": [_vp, ctypes.c_char_p, ctypes.c_char_p, _vp],
        "sgb_block_norm_backward": [_vp, ctypes.c_char_p, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_distill_create": [_out, _i64, _i32, _f32, _f32, _f32],
        "sgb_distill_destroy": [_vp],
        "sgb_distill_workspace_bytes": [_vp, _i64, ctypes.POINTER(_sz)],
        "sgb_distill_forward": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_distill_backward": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_distill_loss_grad": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_penalty_create": [_out, _i64],
        "sgb_penalty_destroy": [_vp],
        "sgb_penalty_workspace_bytes": [_vp, _i64, ctypes.POINTER(_sz)],
        "sgb_penalty_apply": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_vocab_ce_create": [_out, _i32, _i64],
        "sgb_vocab_ce_destroy": [_vp],
        "sgb_vocab_ce_workspace_bytes": [_vp, _i64, _i32, _i32, ctypes.POINTER(_sz)],
        "sgb_vocab_ce_forward": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_vocab_ce_backward": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_vocab_ce_loss_grad": [_vp, ctypes.c_char_p, _vp, _sz, _vp],
        "sgb_dropout_create": [_out, ctypes.c_double],
        "sgb_dropout_destroy": [_vp],
        "sgb_dropout_apply": [_vp, ctypes.c_char_p, _vp],
        "sgb_quant_norm_create": [_out, _i32, _i32, _i32, _f32],
        "sgb_quant_norm_destroy": [_vp],
        "sgb_quant_norm_forward": [_vp, ctypes.c_char_p, _vp]}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = None if _name.endswith("_destroy") else ctypes.c_int

NORM = {"none": 0, "rms": 1, "layer": 2}
CODE = {"int8": (0, torch.int8), "fp8": (1, torch.float8_e4m3fn)}
_DTYPE = {torch.float32: DTYPE["f32"], torch.bfloat16: DTYPE["bf16"], torch.float16: DTYPE["f16"]}

# The argument structs of the headers, packed in C layout.  (A call on one token
# takes a few microseconds in all: a ctypes.Structure would cost more than its
# kernel.)
_NORM_PARAMS = struct.Struct("@4Pi4x")
_NORM_FORWARD = struct.Struct("@6P7q2i")
_NORM_BACKWARD = struct.Struct("@13P10q2i")
_DISTILL = struct.Struct("@10P5qif")
_PENALTY = struct.Struct("@12P7q4i")
_VOCAB_CE = struct.Struct("@9P5q3if")
_DROPOUT = struct.Struct("@4P5q2Q4i")
_QUANT_NORM = struct.Struct("@7P6q4i")


def header_functions(header: str = HEADER) -> list:
    """Names of the functions that include/sgb_lm.h (or another header) declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\**(sgb_\w+)\s*\(", text, re.M)))


def _bad(where: str, what: str):
    raise SgbError(SGB_ERR_INVALID_ARGUMENT, f"{where}: {what}")


# The current stream's handle without the Stream object that
# torch.cuda.current_stream() makes of it (2 us, half a one-token kernel's time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, index) -> int:
    if stream is not None:
        return stream.cuda_stream
    if index < 0:
        return 0
    return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream


def _int(name, v, lo, hi, where) -> int:
    """An integer that the C struct's field holds."""
    v = int(v)
    if not lo <= v < hi:
        _bad(where, f"{name} must be in [{lo}, {hi})")
    return v


class _Handle:
    """Owns a plan handle of the C library, on the device current at creation."""
    _kind = ""

    def _create(self, *args):
        h = _vp()
        name = f"sgb_{self._kind}_create"
        _check(getattr(_lib, name)(ctypes.byref(h), *args), name)
        self.handle = h.value
        # without a GPU a plan checks arguments and its calls end in SGB_ERR_HIP
        self._device = torch.device("cuda", torch.cuda.current_device()) \
            if torch.cuda.is_available() else torch.device("cpu")
        self._index = -1 if self._device.type == "cpu" else self._device.index

    def _matrix(self, name, t, dtype, shape, where):
        """Pointer and row stride of a 2-D argument (None: 0, 0)."""
        if t is None:
            return 0, 0
        if t.shape != shape or t.dtype is not dtype:
            _bad(where, f"{name} must be {list(shape)} {dtype} with adjacent row elements")
        pitch, step = t.stride()
        if step != 1 and shape[1] > 1:
            _bad(where, f"{name} must be {list(shape)} {dtype} with adjacent row elements")
        if t.get_device() != self._index:
            _bad(where, f"{name} must be on {self._device}")
        # the stride of a single row says nothing
        return t.data_ptr(), (pitch if shape[0] > 1 else max(pitch, shape[1]))

    def _vector(self, name, t, dtype, n, where):
        if t is None:
            return 0
        if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
            _bad(where, f"{name} must be contiguous {dtype} of {n} elements")
        if t.get_device() != self._index:
            _bad(where, f"{name} must be on {self._device}")
        return t.data_ptr()

    def close(self):
        if getattr(self, "handle", None):
            getattr(_lib, f"sgb_{self._kind}_destroy")(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Plan(_Handle):
    """A plan whose calls work in a workspace."""

    def workspace_bytes(self, rows: int) -> int:
        n = _sz()
        name = f"sgb_{self._kind}_workspace_bytes"
        _check(getattr(_lib, name)(self.handle, int(rows), ctypes.byref(n)), name)
        return int(n.value)

    def workspace(self, rows: int) -> torch.Tensor:
        """A workspace for calls of up to `rows` rows that follow one another."""
        return torch.empty(self.workspace_bytes(rows), dtype=torch.uint8, device=self._device)

    def device_status(self, workspace, stream=None) -> str:
        """Waits for `stream`; the first error that the last call on `workspace` recorded."""
        out = _i32()
        _check(_lib.sgb_lm_device_status(workspace.data_ptr(), _stream(stream, self._index),
                                         ctypes.byref(out)), "sgb_lm_device_status")
        return sgb_status_string(out.value)

    def _space(self, ws, where):
        if ws is None:
            _bad(where, "workspace is missing")
        if ws.get_device() != self._index or not ws.is_contiguous():
            _bad(where, f"workspace must be contiguous on {self._device}")
        return ws.data_ptr(), ws.numel() * ws.element_size()


class BlockNorm(_Plan):
    """x_out = res_scale * x + gate * post(h), y = pre(x_out), row by row, and
    its backward.  post, pre: "none", "rms" or "layer"; the weights and biases
    (one type: float32, bfloat16 or float16) are read at every call."""
    _kind = "block_norm"

    def __init__(self, D: int, post: str = "rms", pre: str = "rms", post_weight=None,
                 post_bias=None, pre_weight=None, pre_bias=None, post_eps: float = 1e-6,
                 pre_eps: float = 1e-6, res_scale: float = 1.0):
        self.D, self.post, self.pre = int(D), post, pre
        for k in (post, pre):
            if k not in NORM:
                _bad("BlockNorm", f"unknown norm {k!r}")
        self._create(self.D, NORM[post], NORM[pre], post_eps, pre_eps, res_scale)
        self.post_weight, self.post_bias = post_weight, post_bias
        self.pre_weight, self.pre_bias = pre_weight, pre_bias

    def _params(self, where):
        ps = (self.post_weight, self.post_bias, self.pre_weight, self.pre_bias)
        dtype, at = None, [0, 0, 0, 0]
        for i, p in enumerate(ps):
            if p is not None:
                dtype = dtype or p.dtype
                at[i] = self._vector("a parameter", p, dtype, self.D, where)
        dtype = dtype or torch.float32
        if dtype not in _DTYPE:
            _bad(where, f"parameters cannot be {dtype}")
        return _NORM_PARAMS.pack(*at, _DTYPE[dtype])

    def _types(self, x, h, where):
        if x is None or h is None or h.dtype not in _DTYPE or x.dtype not in _DTYPE:
            _bad(where, "x and h must be float32, bfloat16 or float16")
        return h.dtype, x.dtype, x.shape[0], torch.Size((x.shape[0], self.D))

    def _gate(self, gate, rows, rows_per_gate, dt, where):
        if gate is None:
            return 0, 0, 0, None
        rpg = int(rows_per_gate)
        if rpg < 1:
            _bad(where, "rows_per_gate must be at least 1")
        shape = torch.Size(((rows + rpg - 1) // rpg, self.D))
        return (*self._matrix("gate", gate, dt, shape, where), rpg, shape)

    def forward(self, x, h, x_out, y=None, gate=None, rows_per_gate: int = 1, stats=None,
                stream=None) -> None:
        """x, x_out [rows, D] (float32, or h's type), h, y [rows, D], gate
        [ceil(rows / rows_per_gate), D] or None, stats [rows, 4] float32 or
        None (what backward reads).  x_out may be x, y may be h."""
        w = "sgb_block_norm_forward"
        dt, rt, rows, shape = self._types(x, h, w)
        pg, sg, rpg, _ = self._gate(gate, rows, rows_per_gate, dt, w)
        px, sx = self._matrix("x", x, rt, shape, w)
        ph, sh = self._matrix("h", h, dt, shape, w)
        po, so = self._matrix("x_out", x_out, rt, shape, w)
        py, sy = self._matrix("y", y, dt, shape, w)
        st = _lib.sgb_block_norm_forward(
            self.handle, self._params(w),
            _NORM_FORWARD.pack(px, ph, po, py, pg,
                               self._vector("stats", stats, torch.float32, 4 * rows, w),
                               sx, sh, so, sy, sg, rows, rpg, _DTYPE[dt], _DTYPE[rt]),
            _stream(stream, self._index))
        _check(st, w)

    def backward(self, dx_out, dy, x_out, h, stats, dx, dh, gate=None, rows_per_gate: int = 1,
                 d_gate=None, d_post_weight=None, d_post_bias=None, d_pre_weight=None,
                 d_pre_bias=None, workspace=None, stream=None) -> None:
        """Gradients dx, dh, d_gate (the inputs' types) and the parameters'
        (float32) from dx_out and dy; x_out, h, gate and stats are the
        forward's.  dx may be dx_out, dh may be dy or h; sums that are None
        are not computed."""
        w = "sgb_block_norm_backward"
        dt, rt, rows, shape = self._types(dx_out, dh, w)
        pg, sg, rpg, gs = self._gate(gate, rows, rows_per_gate, dt, w)
        pdxo, sdxo = self._matrix("dx_out", dx_out, rt, shape, w)
        pdy, sdy = self._matrix("dy", dy, dt, shape, w)
        px, sx = self._matrix("x_out", x_out, rt, shape, w)
        ph, sh = self._matrix("h", h, dt, shape, w)
        pdx, sdx = self._matrix("dx", dx, rt, shape, w)
        pdh, sdh = self._matrix("dh", dh, dt, shape, w)
        if d_gate is not None and gate is None:
            _bad(w, "d_gate without a gate")
        pdg, sdg = self._matrix("d_gate", d_gate, dt, gs, w)
        f32 = torch.float32
        vec = [self._vector(n, v, f32, self.D, w) for n, v in
               (("d_post_weight", d_post_weight), ("d_post_bias", d_post_bias),
                ("d_pre_weight", d_pre_weight), ("d_pre_bias", d_pre_bias))]
        ws, ws_bytes = self._space(workspace, w)
        st = _lib.sgb_block_norm_backward(
            self.handle, self._params(w),
            _NORM_BACKWARD.pack(pdxo, pdy, px, ph, self._vector("stats", stats, f32, 4 * rows, w),
                                pg, pdx, pdh, pdg, *vec, sdxo, sdy, sx, sh, sg, sdx, sdh, sdg,
                                rows, rpg, _DTYPE[dt], _DTYPE[rt]),
            ws, ws_bytes, _stream(stream, self._index))
        _check(st, w)


class TopkDistill(_Plan):
    """Distillation of a student's logits [rows, V] from the K logits a row
    that a teacher listed: kd_weight T^2 KL(teacher || student) at temperature
    T, plus ce_weight times the labels' cross-entropy."""
    _kind = "distill"

    def __init__(self, V: int, K: int, temperature: float = 1.0, kd_weight: float = 1.0,
                 ce_weight: float = 0.0):
        self.V, self.K = int(V), int(K)
        self._create(self.V, self.K, temperature, kd_weight, ce_weight)

    def _call(self, name, logits, ids, values, loss, stats, grad_loss, grad, grad_scale,
              teacher_lse, labels, row_weights, workspace, stream):
        if logits.dtype not in _DTYPE:
            _bad(name, "logits must be float32, bfloat16 or float16")
        dt, rows = logits.dtype, logits.shape[0]
        full, part = torch.Size((rows, self.V)), torch.Size((rows, self.K))
        pl, sl = self._matrix("logits", logits, dt, full, name)
        pi, si = self._matrix("ids", ids, torch.int64, part, name)
        pv, sv = self._matrix("values", values, torch.float32, part, name)
        pg, sg = self._matrix("grad", grad, dt, full, name)
        f32 = torch.float32
        args = _DISTILL.pack(
            pl, pi, pv, self._vector("teacher_lse", teacher_lse, f32, rows, name),
            self._vector("labels", labels, torch.int64, rows, name),
            self._vector("row_weights", row_weights, f32, rows, name),
            self._vector("loss", loss, f32, rows, name),
            self._vector("stats", stats, f32, 4 * rows, name),
            self._vector("grad_loss", grad_loss, f32, rows, name), pg,
            sl, si, sv, sg, rows, _DTYPE[dt], grad_scale)
        ws, ws_bytes = self._space(workspace, name)
        _check(getattr(_lib, name)(self.handle, args, ws, ws_bytes,
                                   _stream(stream, self._index)), name)

    def forward(self, logits, ids, values, loss, stats=None, teacher_lse=None, labels=None,
                row_weights=None, workspace=None, stream=None) -> None:
        """loss [rows] float32; stats [rows, 4] float32 where a backward is to
        follow.  ids [rows, K] int64 (negative: not listed), values [rows, K]
        float32, teacher_lse / row_weights [rows] float32 or None, labels
        [rows] int64 (negative: none)."""
        self._call("sgb_distill_forward", logits, ids, values, loss, stats, None, None, 0.0,
                   teacher_lse, labels, row_weights, workspace, stream)

    def backward(self, logits, ids, values, stats, grad_loss, grad, grad_scale: float = 1.0,
                 teacher_lse=None, labels=None, row_weights=None, workspace=None,
                 stream=None) -> None:
        """grad [rows, V] in the logits' type: grad_scale * grad_loss[row] *
        d loss[row] / d logits (grad_loss None: 1), from forward's stats."""
        self._call("sgb_distill_backward", logits, ids, values, None, stats, grad_loss, grad,
                   grad_scale, teacher_lse, labels, row_weights, workspace, stream)

    def loss_grad(self, logits, ids, values, loss, grad, grad_scale: float = 1.0,
                  teacher_lse=None, labels=None, row_weights=None, workspace=None,
                  stream=None) -> None:
        """forward and backward in one go."""
        self._call("sgb_distill_loss_grad", logits, ids, values, loss, None, None, grad,
                   grad_scale, teacher_lse, labels, row_weights, workspace, stream)


class LogitsPenalty(_Plan):
    """Repetition, frequency and presence penalties, biases and grammar masks
    on logits [rows, vocab] before sampling."""
    _kind = "penalty"

    def __init__(self, vocab: int):
        self.vocab = int(vocab)
        self._create(self.vocab)

    def apply(self, logits, out, tokens=None, prompt_lens=None, lens=None, repetition=None,
              frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None,
              mask_index=None, workspace=None, stream=None) -> None:
        """out (may be logits) [rows, vocab]; tokens [rows, max_tokens] int32,
        of which a row has lens[row] (None: all), the first prompt_lens[row]
        (None: none) a prompt; repetition, frequency, presence [rows] float32;
        bias_ids [rows, n] int32 (negative: none) with bias_values float32;
        mask [masks, >= ceil(vocab / 32)] int32, a bit a token (set: allowed),
        mask_index [rows] int32 (negative: unmasked; None: row r has mask r)."""
        w = "sgb_penalty_apply"
        if logits.dtype not in _DTYPE:
            _bad(w, "logits must be float32, bfloat16 or float16")
        dt, rows = logits.dtype, logits.shape[0]
        full = torch.Size((rows, self.vocab))
        f32, i32 = torch.float32, torch.int32
        pl, sl = self._matrix("logits", logits, dt, full, w)
        po, so = self._matrix("out", out, dt, full, w)
        L = n = masks = 0
        pt = st_ = pbi = sbi = pb = sb = pm = sm = 0
        for name, t in (("tokens", tokens), ("bias_ids", bias_ids), ("mask", mask)):
            if t is not None and t.dim() != 2:
                _bad(w, f"{name} must be a matrix")
        if tokens is not None:
            L = tokens.shape[1]
            pt, st_ = self._matrix("tokens", tokens, i32, torch.Size((rows, L)), w)
        if bias_values is not None and bias_ids is None:
            _bad(w, "bias_values without bias_ids")
        if bias_ids is not None:
            n = bias_ids.shape[1]
            pbi, sbi = self._matrix("bias_ids", bias_ids, i32, torch.Size((rows, n)), w)
            pb, sb = self._matrix("bias_values", bias_values, f32, torch.Size((rows, n)), w)
        if mask is not None:
            masks, words = mask.shape
            if words < (self.vocab + 31) // 32:
                _bad(w, f"mask must have {(self.vocab + 31) // 32} words a row")
            pm, sm = self._matrix("mask", mask, i32, mask.shape, w)
            if masks == 0:   # no address, but a set all the same: every index is past its end
                if mask_index is None and rows:
                    _bad(w, "mask must have a row for each of the logits' without mask_index")
                pm = self._vector("mask_index", mask_index, i32, rows, w)
        args = _PENALTY.pack(
            pl, po, pt, self._vector("prompt_lens", prompt_lens, i32, rows, w),
            self._vector("lens", lens, i32, rows, w),
            self._vector("repetition", repetition, f32, rows, w),
            self._vector("frequency", frequency, f32, rows, w),
            self._vector("presence", presence, f32, rows, w), pbi, pb, pm,
            self._vector("mask_index", mask_index, i32, rows, w) if mask is not None else 0,
            sl, so, st_, sbi, sb, sm, rows, L, n, masks, _DTYPE[dt])
        ws, ws_bytes = self._space(workspace, w)
        _check(_lib.sgb_penalty_apply(self.handle, args, ws, ws_bytes,
                                      _stream(stream, self._index)), w)


class VocabCrossEntropy(_Plan):
    """Cross-entropy of the head's product hidden @ weight.T over a vocabulary
    of V tokens, D columns, with its gradients, without a matrix of logits:
    the workspace holds the exponentials of a chunk of rows where there are
    gradients, and is a few GiB at most (4096 columns, 131072 tokens, bf16:
    3.0 GiB for 8192 rows, 5.0 for any more, 0.6 for the loss alone)."""
    _kind = "vocab_ce"

    def __init__(self, D: int, V: int):
        self.D = _int("D", D, -2**31, 2**31, "VocabCrossEntropy")
        self.V = _int("V", V, -2**63, 2**63, "VocabCrossEntropy")
        self._create(self.D, self.V)

    def workspace_bytes(self, rows: int, dtype=torch.bfloat16, gradient: bool = True,
                        exact: bool = False) -> int:
        w = "sgb_vocab_ce_workspace_bytes"
        if dtype not in _DTYPE:
            _bad(w, "dtype must be float32, bfloat16 or float16")
        n = _sz()
        _check(_lib.sgb_vocab_ce_workspace_bytes(self.handle, _int("rows", rows, -2**63, 2**63, w),
                                                 _DTYPE[dtype], (1 + bool(exact)) * bool(gradient),
                                                 ctypes.byref(n)), w)
        return int(n.value)

    def workspace(self, rows: int, dtype=torch.bfloat16, gradient: bool = True,
                  exact: bool = False) -> torch.Tensor:
        """A workspace for calls of up to `rows` rows of that type that follow
        one another; without gradient for forward alone, with exact for calls
        for exact gradients as well."""
        return torch.empty(self.workspace_bytes(rows, dtype, gradient, exact), dtype=torch.uint8,
                           device=self._device)

    def _call(self, name, hidden, weight, labels, loss, lse, grad_loss, d_hidden, d_weight,
              grad_scale, accumulate, exact, row_weights, workspace, stream):
        if hidden.dtype not in _DTYPE:
            _bad(name, "hidden must be float32, bfloat16 or float16")
        dt, rows = hidden.dtype, hidden.shape[0]
        full, head = torch.Size((rows, self.D)), torch.Size((self.V, self.D))
        f32 = torch.float32
        wt = dt if d_weight is None else d_weight.dtype
        if wt is not dt and wt is not f32:
            _bad(name, f"d_weight must be {dt} or float32")
        ph, sh = self._matrix("hidden", hidden, dt, full, name)
        pw, sw = self._matrix("weight", weight, dt, head, name)
        pdh, sdh = self._matrix("d_hidden", d_hidden, dt, full, name)
        pdw, sdw = self._matrix("d_weight", d_weight, wt, head, name)
        args = _VOCAB_CE.pack(
            ph, pw, self._vector("labels", labels, torch.int64, rows, name),
            self._vector("row_weights", row_weights, f32, rows, name),
            self._vector("loss", loss, f32, rows, name), self._vector("lse", lse, f32, rows, name),
            self._vector("grad_loss", grad_loss, f32, rows, name), pdh, pdw,
            sh, sw, sdh, sdw, rows, _DTYPE[dt], _DTYPE[wt], bool(accumulate) + 2 * bool(exact),
            grad_scale)
        ws, ws_bytes = self._space(workspace, name)
        _check(getattr(_lib, name)(self.handle, args, ws, ws_bytes,
                                   _stream(stream, self._index)), name)

    def forward(self, hidden, weight, labels, loss, lse=None, row_weights=None, workspace=None,
                stream=None) -> None:
        """loss [rows] float32, and lse [rows] float32 where a backward is to
        follow.  hidden [rows, D], weight [V, D] (of one type), labels [rows]
        int64 (negative: none), row_weights [rows] float32 or None."""
        self._call("sgb_vocab_ce_forward", hidden, weight, labels, loss, lse, None, None, None,
                   0.0, False, False, row_weights, workspace, stream)

    def backward(self, hidden, weight, labels, lse, grad_loss=None, d_hidden=None, d_weight=None,
                 grad_scale: float = 1.0, accumulate: bool = False, row_weights=None,
                 workspace=None, stream=None, exact: bool = False) -> None:
        """d_hidden [rows, D] in hidden's type and d_weight [V, D] in weight's
        type or float32 (None: not wanted) of grad_scale * sum(grad_loss *
        loss), from forward's lse; accumulate: d_weight is added to; exact: of
        16-bit types, the logits' gradient is multiplied with what its rounding
        leaves, as it always is in calls of up to 128 rows: the gradients' error
        is their own rounding alone, and their products take twice as long."""
        self._call("sgb_vocab_ce_backward", hidden, weight, labels, None, lse, grad_loss, d_hidden,
                   d_weight, grad_scale, accumulate, exact, row_weights, workspace, stream)

    def loss_grad(self, hidden, weight, labels, loss, d_hidden=None, d_weight=None,
                  grad_scale: float = 1.0, accumulate: bool = False, lse=None, row_weights=None,
                  workspace=None, stream=None, exact: bool = False) -> None:
        """forward and backward (without grad_loss) in one go: one product less."""
        self._call("sgb_vocab_ce_loss_grad", hidden, weight, labels, loss, lse, None, d_hidden,
                   d_weight, grad_scale, accumulate, exact, row_weights, workspace, stream)


class Dropout(_Handle):
    """Dropout with probability p (to 2^-16) from a counter-based generator:
    the mask is a function of (seed, offset, row, column) and never stored."""
    _kind = "dropout"

    def __init__(self, p: float):
        self.p = float(p)
        self._create(self.p)

    def _call(self, x, out, seed, offset, residual, state, first_row, stream):
        w = "sgb_dropout_apply"
        if x.dtype not in _DTYPE or out is None or out.dtype not in _DTYPE:
            _bad(w, "x and out must be float32, bfloat16 or float16")
        if x.dim() != 2:
            _bad(w, "x must be a matrix")
        shape, ot = x.shape, out.dtype
        px, sx = self._matrix("x", x, x.dtype, shape, w)
        pr, sr = self._matrix("residual", residual, ot, shape, w)
        po, so = self._matrix("out", out, ot, shape, w)
        args = _DROPOUT.pack(px, pr, po, self._vector("state", state, torch.int64, 2, w), sx, sr, so,
                             shape[0], _int("first_row", first_row, 0, 2**62, w),
                             _int("seed", seed, 0, 2**64, w), _int("offset", offset, 0, 2**64, w),
                             _int("columns", shape[1], 0, 2**31, w), _DTYPE[x.dtype], _DTYPE[ot], 0)
        _check(_lib.sgb_dropout_apply(self.handle, args, _stream(stream, self._index)), w)

    def forward(self, x, out, seed: int = 0, offset: int = 0, residual=None, state=None,
                first_row: int = 0, stream=None) -> None:
        """out = residual + dropped x; x, out [rows, columns], residual in
        out's type (x's, or float32) or None (0; out then in x's type).  out
        may be x or residual.  state: two int64 on the device, the seed and
        what is added to the offset, read when the kernel runs."""
        self._call(x, out, seed, offset, residual, state, first_row, stream)

    def backward(self, d_out, dx, seed: int = 0, offset: int = 0, state=None, first_row: int = 0,
                 stream=None) -> None:
        """dx (may be d_out) from d_out, in one type, under the forward's mask;
        the residual's gradient is d_out."""
        self._call(d_out, dx, seed, offset, None, state, first_row, stream)


class QuantNorm(_Handle):
    """x_out = x + h and the codes of rms(x_out) * weight in 8 bits ("int8", or
    "fp8": e4m3) with a scale a row (group 0) or a group of columns."""
    _kind = "quant_norm"

    def __init__(self, D: int, weight=None, form: str = "int8", group: int = 0, eps: float = 1e-6):
        w = "QuantNorm"
        if form not in CODE:
            _bad(w, f"unknown form {form!r}")
        self.D, self.group = _int("D", D, -2**31, 2**31, w), _int("group", group, -2**31, 2**31, w)
        self.form, self.weight = form, weight
        self._code, self._type = CODE[form]
        self._create(self.D, self._code, self.group, eps)
        self.groups = -(-self.D // self.group) if self.group else 1

    def forward(self, h, q, scales, x=None, x_out=None, stats=None, stream=None) -> None:
        """h [rows, D]; x, x_out [rows, D] (float32, or h's type) or None; q
        [rows, D] int8 or float8_e4m3fn; scales [rows, groups] float32; stats
        [rows, 4] float32 or None (what a BlockNorm with post="none",
        pre="rms" reads in its backward).  x_out may be x, or h."""
        w = "sgb_quant_norm_forward"
        if h.dtype not in _DTYPE:
            _bad(w, "h must be float32, bfloat16 or float16")
        if self.weight is None or self.weight.dtype not in _DTYPE:
            _bad(w, "weight must be float32, bfloat16 or float16")
        dt, rows, f32 = h.dtype, h.shape[0], torch.float32
        rt = x.dtype if x is not None else x_out.dtype if x_out is not None else dt
        if rt not in _DTYPE:
            _bad(w, "x and x_out must be float32 or h's type")
        shape = torch.Size((rows, self.D))
        ph, sh = self._matrix("h", h, dt, shape, w)
        px, sx = self._matrix("x", x, rt, shape, w)
        po, so = self._matrix("x_out", x_out, rt, shape, w)
        pq, sq = self._matrix("q", q, self._type, shape, w)
        ps, ss = self._matrix("scales", scales, f32, torch.Size((rows, self.groups)), w)
        args = _QUANT_NORM.pack(
            ph, px, po, self._vector("weight", self.weight, self.weight.dtype, self.D, w), pq, ps,
            self._vector("stats", stats, f32, 4 * rows, w), sh, sx, so, sq, ss, rows, _DTYPE[dt],
            _DTYPE[rt], _DTYPE[self.weight.dtype], 0)
        _check(_lib.sgb_quant_norm_forward(self.handle, args, _stream(stream, self._index)), w)
