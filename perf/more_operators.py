"""More token-model operators, case by case: cross-entropy of the head product
over a large vocabulary (loss, gradients), dropout from a counter-based
generator (forward, backward), rms norm with the residual's addition and an
8-bit output.

`own` False: `run` computes an operator in plain torch operations, in fp32,
rounded once at the end.  `own` True: `run` calls the library's entry points
(`sparse_gradient_backward_amd.lm`).  Both take what `prepare` returns.
`exact` evaluates the definitions in fp64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
VOCAB = 131072   # the token-embedding workload's vocabulary; its rows are 4096 wide
CODES = {"int8": (torch.int8, 127.0), "fp8": (torch.float8_e4m3fn, 448.0)}


# ------------------------------------------------------------------ cases

def _head(name, rows, D, V, way, dt):
    """way: loss; both (loss and gradients in one call); split (a forward, then
    a backward under a gradient from above)."""
    return dict(name=name, op="head", rows=rows, D=D, V=V, way=way, dtype=dt)


def _drop(name, rows, D, way, dt, res, p, pad=0):
    """res: the residual's type, or none; pad: columns of a wider buffer
    between one row of x and the next."""
    return dict(name=name, op="drop", rows=rows, D=D, way=way, dtype=dt, res=res, p=p, pad=pad)


def _quant(name, rows, D, dt, res, form, group):
    """res: the residual's type, or none; group: columns to a scale (0: a row)."""
    return dict(name=name, op="quant", rows=rows, D=D, dtype=dt, res=res, form=form, group=group)


def listed():
    return [
        # the example model's training step
        _head("head_small", 512, 256, 2000, "both", "f32"),
        # a training step over the token-embedding workload's vocabulary
        _head("head_train", 8192, 4096, VOCAB, "both", "bf16"),
        # loss first, gradients later under a gradient from above; odd sizes
        _head("head_odd", 1021, 1001, 50021, "split", "f16"),
        # evaluation of a short text: the loss alone
        _head("head_eval", 512, 4096, VOCAB, "loss", "bf16"),
        # the example model's embedding rows
        _drop("drop_small", 512, 256, "fwd", "f32", "none", 0.1),
        # a training step of 8 x 4096 tokens: a block's output onto the residual stream
        _drop("drop_train", 32768, 4096, "fwd", "bf16", "bf16", 0.1),
        # its backward
        _drop("drop_back", 32768, 4096, "bwd", "bf16", "none", 0.1),
        # odd sizes, rows of a wider buffer, fp32 residual stream
        _drop("drop_odd", 3001, 1001, "fwd", "f16", "f32", 0.25, 7),
        # one token being generated: a code row and one scale
        _quant("quant_token", 1, 4096, "bf16", "bf16", "int8", 0),
        # a prompt on an fp32 residual stream, a scale to 128 columns
        _quant("quant_prompt", 8192, 4096, "bf16", "f32", "fp8", 128),
        # odd sizes; the last group of a row is a short one
        _quant("quant_odd", 3001, 1001, "f16", "f16", "fp8", 64),
        # the norm before the head: no residual; a large batch of prompts
        _quant("quant_large", 32768, 4096, "bf16", "none", "fp8", 0),
    ]


def draw(rng):
    def log(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if rng.random() < 0.5:      # rounded to what vector widths like, or left as it falls
            m = 64 if n >= 640 else 8 if n >= 16 else 1
            n = n // m * m
        return max(lo, min(hi, n))

    c = _draw(rng, log)
    del c["name"]
    return c


def _draw(rng, log):
    op = rng.choice(("head", "drop", "quant"))
    dt = rng.choice(("f32", "bf16", "f16"))
    if op == "head":
        D, V = log(64, 4096), log(1000, VOCAB)
        # an fp32 product costs several times one of 16 bits
        rows = log(1, min(8192, 8192 * 4096 * VOCAB // ((8 if dt == "f32" else 1) * D * V)))
        return _head("", rows, D, V, rng.choice(("both", "both", "split", "loss")), dt)
    D = log(64, 8192)
    rows = log(1, min(32768, 32768 * 4096 // ((2 if dt == "f32" else 1) * D)))
    if op == "drop":
        way = rng.choice(("fwd", "bwd"))
        res = rng.choice(("none", dt)) if way == "fwd" else "none"
        return _drop("", rows, D, way, dt, res, rng.choice((0.05, 0.1, 0.2, 0.5)),
                     rng.choice((0, 0, 8, 3)))
    form = rng.choice(("int8", "fp8", "fp8"))
    group = rng.choice((0, 0, 32, 64, 128))
    if form == "int8" and group:
        D = max(group, D // group * group)
    return _quant("", rows, D, dt, rng.choice(("none", dt, dt)), form, group)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    return {"head": _prepare_head, "drop": _prepare_drop, "quant": _prepare_quant}[case["op"]](
        case, g, seed)


def _normal(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _prepare_head(c, g, seed):
    R, D, V, dt = c["rows"], c["D"], c["V"], DTYPES[c["dtype"]]
    s = dict(case=c, hidden=_normal(g, R, D, dtype=dt))          # what a norm returns
    s["weight"] = torch.empty(V, D, dtype=dt, device="cuda")
    for a in range(0, V, 1 << 16):
        b = min(V, a + (1 << 16))
        s["weight"][a:b] = _normal(g, b - a, D, std=2.0 / math.sqrt(D))
    # Zipf-like labels, as in text; some tokens have none, some are padding
    u = torch.rand(R, generator=g, device="cuda", dtype=torch.float64)
    s["labels"] = (torch.exp(u * math.log(V)) - 1).long().clamp_(0, V - 1)
    s["labels"][torch.rand(R, generator=g, device="cuda") < 0.1] = -1
    s["weights"] = torch.rand(R, generator=g, device="cuda") + 0.5
    s["weights"][torch.rand(R, generator=g, device="cuda") < 0.1] = 0
    s["labels"][0], s["weights"][0] = V // 2, 1.0
    s["loss"] = torch.empty(R, device="cuda")
    s["lse"] = torch.empty(R, device="cuda")
    s["d_hidden"] = s["d_weight"] = None
    # fp16 gradients are kept in range by a scale on the loss
    s["scale"] = 16.0 if c["dtype"] == "f16" else 1.0 / R
    if c["way"] != "loss":
        s["d_hidden"], s["d_weight"] = torch.empty_like(s["hidden"]), torch.empty_like(s["weight"])
    if c["way"] == "split":
        s["grad_loss"] = torch.rand(R, generator=g, device="cuda") + 0.5
    if own:
        from sparse_gradient_backward_amd import lm
        s["head"] = lm.VocabCrossEntropy(D, V)
        s["ws"] = s["head"].workspace(R, dt, gradient=c["way"] != "loss")
    return s


def _prepare_drop(c, g, seed):
    R, D, dt = c["rows"], c["D"], DTYPES[c["dtype"]]
    s = dict(case=c, seed=(7919 * seed + 11) << 20 | 5, offset=seed % 1000)
    s["x"] = _normal(g, R, D + c["pad"], dtype=dt)[:, :D]
    s["res"] = None if c["res"] == "none" else _normal(g, R, D, std=3.0, dtype=DTYPES[c["res"]])
    s["out"] = torch.empty(R, D, dtype=dt if s["res"] is None else s["res"].dtype, device="cuda")
    if own:
        from sparse_gradient_backward_amd import lm
        s["drop"] = lm.Dropout(c["p"])
    return s


def _prepare_quant(c, g, seed):
    R, D, dt = c["rows"], c["D"], DTYPES[c["dtype"]]
    s = dict(case=c, eps=1e-6, h=_normal(g, R, D, std=0.8, dtype=dt))
    # a few columns are much larger than the others, as in trained models
    wide = torch.rand(D, generator=g, device="cuda") < 0.01
    s["h"][:, wide] *= 10
    s["x"] = None if c["res"] == "none" else _normal(g, R, D, std=3.0, dtype=DTYPES[c["res"]])
    s["w"] = _normal(g, D, std=0.2, mean=1.0)
    s["x_out"] = None if s["x"] is None else torch.empty_like(s["x"])
    n = c["group"] or D
    s["scales"] = torch.empty(R, (D + n - 1) // n, device="cuda")
    s["q"] = torch.empty(R, D, dtype=CODES[c["form"]][0], device="cuda")
    # int8 codes are read as the values they stand for, in 16 bits
    s["y"] = torch.empty(R, D, dtype=torch.bfloat16, device="cuda") if c["form"] == "int8" else None
    if own:
        from sparse_gradient_backward_amd import lm
        s["norm"] = lm.QuantNorm(D, weight=s["w"], form=c["form"], group=c["group"], eps=s["eps"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op, way = s["case"]["op"], s["case"].get("way")
    if own:
        return {"head": _own_head, "drop": _own_drop, "quant": _own_quant}[op](s, way)
    return {"head": _plain_head, "drop": _plain_drop, "quant": _plain_quant}[op](s, way)


def _own_head(s, way):
    h, args = s["head"], (s["hidden"], s["weight"], s["labels"])
    kw = dict(row_weights=s["weights"], workspace=s["ws"])
    if way == "both":
        h.loss_grad(*args, s["loss"], s["d_hidden"], s["d_weight"], grad_scale=s["scale"],
                    lse=s["lse"], **kw)
    else:
        h.forward(*args, s["loss"], lse=s["lse"], **kw)
        if way == "split":
            h.backward(*args, s["lse"], s["grad_loss"], s["d_hidden"], s["d_weight"],
                       grad_scale=s["scale"], **kw)
    return dict(loss=s["loss"], lse=s["lse"], d_hidden=s["d_hidden"], d_weight=s["d_weight"])


def _own_drop(s, way):
    if way == "fwd":
        s["drop"].forward(s["x"], s["out"], s["seed"], s["offset"], residual=s["res"])
    else:
        s["drop"].backward(s["x"], s["out"], s["seed"], s["offset"])
    return s["out"]


def _own_quant(s, way):
    s["norm"].forward(s["h"], s["q"], s["scales"], x=s["x"], x_out=s["x_out"])
    return _quant_outputs(s)


def _quant_outputs(s):
    c = s["case"]
    values = s["q"]
    if c["form"] == "int8":
        R, D, n = c["rows"], c["D"], c["group"] or c["D"]
        torch.mul(s["q"].view(R, D // n, n), s["scales"][:, :, None], out=s["y"].view(R, D // n, n))
        values = s["y"]
    return dict(x_out=s["x_out"], values=values, scales=s["scales"])


def _plain_head(s, way):
    x, w = s["hidden"].float(), s["weight"].float()
    logits = x @ w.t()
    top = logits.max(1, keepdim=True).values
    on = s["labels"] >= 0
    label = s["labels"].clamp(min=0)[:, None]
    said = logits.gather(1, label)
    e = logits.sub_(top).exp_()
    total = e.sum(1, keepdim=True)
    factor = torch.where(on, s["weights"], 0)
    lse = top + total.log()
    out = dict(loss=torch.where(factor != 0, factor * (lse - said)[:, 0], 0), lse=lse[:, 0],
               d_hidden=None, d_weight=None)
    if way == "loss":
        return out
    above = factor * s["scale"] * (s["grad_loss"] if way == "split" else 1)
    g = e.mul_((above / total[:, 0])[:, None])
    g.scatter_add_(1, label, -above[:, None])
    out["d_hidden"], out["d_weight"] = (g @ w).to(s["hidden"].dtype), (g.t() @ x).to(s["weight"].dtype)
    return out


def _draws(s, rows, D):
    """16 random bits for each element: Philox4x32-10 with the seed as key and
    the counter (column / 8, row, 2^31, offset); eight elements take the low
    and the high half of each of its four words in turn."""
    low = 0xFFFFFFFF
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    device = s["x"].device
    groups = (D + 7) // 8
    a = torch.arange(groups, device=device).expand(rows, groups)
    b = torch.arange(rows, device=device)[:, None].expand(rows, groups)
    c = torch.full((1, 1), 1 << 31, device=device)
    d = torch.full((1, 1), s["offset"] & low, device=device)
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57      # the low 64 bits of each product
        a, b, c, d = ((q >> 32) & low) ^ b ^ k0, q & low, ((p >> 32) & low) ^ d ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([t.expand(rows, groups) for t in (a, b, c, d)], 2)
    halves = torch.stack([words & 0xFFFF, words >> 16], 3)
    return halves.reshape(rows, groups * 8)[:, :D]


def _plain_drop(s, way):
    c = s["case"]
    cut = round(c["p"] * 65536)
    y = torch.where(_draws(s, c["rows"], c["D"]) >= cut, s["x"].float() * (65536 / (65536 - cut)), 0)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["out"].dtype)


def _plain_quant(s, way):
    c = s["case"]
    R, D, n = c["rows"], c["D"], c["group"] or c["D"]
    t = s["h"].float()
    if s["x"] is not None:
        t = t + s["x"].float()
        s["x_out"].copy_(t)
    v = t * (t.square().mean(1, keepdim=True) + s["eps"]).rsqrt() * s["w"]
    groups = s["scales"].shape[1]
    v = torch.nn.functional.pad(v, (0, groups * n - D)).view(R, groups, n)
    most = CODES[c["form"]][1]
    scale = v.abs().amax(2) / most
    there = scale >= 2.0 ** -126
    s["scales"].copy_(torch.where(there, scale, 0))
    code = torch.where(there[:, :, None], v / scale[:, :, None], 0).clamp(-most, most)
    code = code.view(R, groups * n)[:, :D]
    s["q"].copy_(code.round() if c["form"] == "int8" else code)
    return _quant_outputs(s)


# ------------------------------------------------------------------ work of one pass

def work(case):
    c = case
    R, D, el = c["rows"], c["D"], SIZE[c["dtype"]]
    res = SIZE.get(c.get("res"), 0)
    if c["op"] == "head":
        V, grad = c["V"], c["way"] != "loss"
        return dict(bytes=(R * D + V * D) * el * (1 + grad) + R * 16, flops=2 * R * D * V * (1 + 2 * grad))
    if c["op"] == "drop":
        return dict(bytes=R * D * (el + res + (res or el)), flops=12 * R * D)
    return dict(bytes=R * D * (el + 2 * res + 1) + 4 * R * ((D - 1) // (c["group"] or D) + 1) + 4 * D,
                flops=8 * R * D)


# ------------------------------------------------------------------ the definitions in fp64

def exact(case, seed):
    s = prepare(case, seed)
    return {"head": _exact_head, "drop": _exact_drop, "quant": _exact_quant}[case["op"]](s)


def _exact_head(s):
    c = s["case"]
    R, V = c["rows"], c["V"]
    w = s["weight"].double()
    grad = c["way"] != "loss"
    losses, lses, dh, dw = [], [], [], torch.zeros_like(w) if grad else None
    step = max(1, min(R, (1 << 28) // V))
    for a in range(0, R, step):
        r = slice(a, min(R, a + step))
        x, labels, f = s["hidden"][r].double(), s["labels"][r], s["weights"][r].double()
        logp = torch.mm(x, w.t())
        lses.append(torch.logsumexp(logp, 1))
        logp -= lses[-1][:, None]
        has = torch.nonzero(labels >= 0)[:, 0]
        loss = torch.zeros_like(f)
        loss[has] = -f[has] * logp[has, labels[has]]
        losses.append(loss)
        if grad:
            up = torch.zeros_like(f)
            up[has] = f[has] * s["scale"]
            if c["way"] == "split":
                up = up * s["grad_loss"][r].double()
            g = logp.exp_()
            g[has, labels[has]] -= 1
            g *= up[:, None]
            dh.append(torch.mm(g, w))
            dw.addmm_(g.t(), x)
            del g
        del logp
    return dict(loss=torch.cat(losses), lse=torch.cat(lses), d_hidden=torch.cat(dh) if grad else None, d_weight=dw)


def _exact_drop(s):
    c = s["case"]
    R, D = c["rows"], c["D"]
    cut, out = round(c["p"] * 65536), []
    u32, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for a in range(0, R, 4096):
        rows = np.arange(a, min(R, a + 4096), dtype=np.uint64)[:, None]
        x = [np.broadcast_to(v, (len(rows), (D + 7) // 8)) for v in
             (np.arange((D + 7) // 8, dtype=np.uint64)[None], rows, np.uint64(1 << 31),
              np.uint64(s["offset"]))]
        for i in range(10):
            key = [np.uint64(((s["seed"] >> 32 * j & 0xFFFFFFFF) + i * bump) & 0xFFFFFFFF)
                   for j, bump in ((0, 0x9E3779B9), (1, 0xBB67AE85))]
            m = [x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)]
            x = [m[1] >> half ^ x[1] ^ key[0], m[1] & u32, m[0] >> half ^ x[3] ^ key[1], m[0] & u32]
        bits = np.stack(x, 2).astype("<u4").view("<u2").reshape(len(rows), -1)[:, :D]
        kept = torch.from_numpy(bits >= cut).cuda().double()
        v = s["x"][a:a + 4096].double() * kept / (1 - cut / 65536)
        out.append(v if s["res"] is None else v + s["res"][a:a + 4096].double())
    return torch.cat(out)


def _exact_quant(s):
    c = s["case"]
    R, D, n = c["rows"], c["D"], c["group"] or c["D"]
    most = CODES[c["form"]][1]
    t = s["h"].double() if s["x"] is None else s["h"].double() + s["x"].double()
    v = t / torch.sqrt(torch.linalg.vector_norm(t, dim=1, keepdim=True) ** 2 / D + s["eps"]) * s["w"]
    values, scales = torch.empty_like(v), []
    for a in range(0, D, n):
        part = v[:, a:a + n]
        scale = part.abs().max(1, keepdim=True).values / most
        code = part / scale
        if c["form"] == "int8":
            values[:, a:a + n] = code.round() * scale
        else:   # three bits after the first, the smallest step 2^-9
            step = torch.exp2(torch.floor(torch.log2(code.abs().clamp(min=2.0 ** -6))) - 3)
            values[:, a:a + n] = (code / step).round() * step
        scales.append(scale)
    return dict(x_out=None if s["x"] is None else t, values=values, scales=torch.cat(scales, 1))
