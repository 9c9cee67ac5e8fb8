"""The token-model operators, case by case: block norms (forward and backward),
top-K distillation (loss, gradient) and logits penalties.

`own` False: `run` computes an operator in plain torch operations, in fp32,
rounded once at the end.  `own` True: `run` calls the library's entry points
(`sparse_gradient_backward_amd.lm`).  Both take what `prepare` returns.
`exact` evaluates the definitions in fp64, the gradients by differentiating
them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
VOCAB = 131072   # the token-embedding workload's vocabulary; its rows are 4096 wide


# ------------------------------------------------------------------ cases

def _norm(name, rows, D, way, res, dt, post, pre, bias, gate, scale=1.0):
    """gate: rows that share one gate row (0: no gate; rows: one for all)."""
    return dict(name=name, op="norm", rows=rows, D=D, way=way, res=res, dtype=dt, post=post,
                pre=pre, bias=bias, gate=gate, scale=scale)


def _distill(name, rows, V, K, way, dt, T, kd, ce, tail):
    return dict(name=name, op="distill", rows=rows, V=V, K=K, way=way, dtype=dt, T=T, kd=kd,
                ce=ce, tail=tail)


def _penalty(name, rows, V, tokens, biases, masks, dt):
    """tokens: the longest sequence so far; masks: distinct grammar states
    (0: no mask), shared by the rows."""
    return dict(name=name, op="penalty", rows=rows, V=V, tokens=tokens, biases=biases,
                masks=masks, dtype=dt)


def listed():
    return [
        # one token being generated: between two blocks, everything on
        _norm("norm_token", 1, 4096, "fwd", "bf16", "bf16", "rms", "rms", False, 1),
        # a prompt, fp32 residual stream (what the embedding forward returns),
        # a gate per sample of 1024 tokens, layer norms with biases
        _norm("norm_prompt", 8192, 4096, "fwd", "f32", "bf16", "layer", "layer", True, 1024),
        # training step of 8 x 4096 tokens: rms norms, one learned gate row
        _norm("norm_train", 32768, 4096, "bwd", "bf16", "bf16", "rms", "rms", False, 32768, 0.5),
        # odd width and rows, a gate of its own for every token
        _norm("norm_odd", 3001, 1001, "bwd", "f16", "f16", "layer", "rms", True, 1),
        # a small student on a small batch, fp32 logits
        _distill("distill_small", 24, 32000, 20, "both", "f32", 2.0, 1.0, 0.0, False),
        # a training step's logits: loss and gradient in one go, teacher's
        # tail mass kept, mixed with the labels' cross-entropy
        _distill("distill_train", 4096, VOCAB, 64, "both", "bf16", 1.0, 0.7, 0.3, True),
        # loss first, gradient later under a gradient from above; odd vocabulary
        _distill("distill_odd", 1021, 50021, 33, "split", "f16", 1.5, 0.5, 0.5, True),
        # evaluation: the loss alone
        _distill("distill_eval", 512, VOCAB, 64, "loss", "bf16", 1.0, 1.0, 0.0, False),
        # one sequence being generated, no grammar
        _penalty("penalty_token", 1, 32000, 700, 0, 0, "f32"),
        # a serving batch, part of it under grammars
        _penalty("penalty_batch", 64, VOCAB, 4096, 16, 8, "bf16"),
        # odd vocabulary, few long sequences
        _penalty("penalty_long", 9, 50021, 60001, 5, 3, "f16"),
        # the largest batch: fp32 logits, long biases
        _penalty("penalty_large", 512, VOCAB, 8192, 300, 64, "f32"),
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
    op = rng.choice(("norm", "distill", "penalty"))
    dt = rng.choice(("f32", "bf16", "f16"))
    if op == "norm":
        D = log(64, 8192)
        rows = log(1, min(32768, 32768 * 4096 // (4 * D) if dt == "f32" else 32768 * 4096 // (2 * D)))
        res = rng.choice((dt, "f32"))
        post, pre = rng.choice((("rms", "rms"), ("layer", "layer"), ("none", "rms"),
                                ("rms", "none"), ("none", "layer")))
        gate = rng.choice((0, 1, rows, max(1, rows // rng.choice((2, 4, 7)))))
        return _norm("", rows, D, rng.choice(("fwd", "bwd")), res, dt, post, pre,
                     rng.random() < 0.5, gate, rng.choice((1.0, 0.5)))
    if op == "distill":
        V = log(1000, VOCAB)
        rows = log(1, min(4096, 4096 * VOCAB // ((2 if dt == "f32" else 1) * V)))
        ce = rng.choice((0.0, 0.3))
        return _distill("", rows, V, log(1, 128), rng.choice(("both", "both", "split", "loss")),
                        dt, rng.choice((1.0, 2.0, 1.5)), 1.0 - ce, ce, rng.random() < 0.5)
    return _penalty("", log(1, 512), log(1000, VOCAB), log(1, 8192), rng.choice((0, 7, 64, 300)),
                    rng.choice((0, 1, 16, 64)), dt)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    return {"norm": _prepare_norm, "distill": _prepare_distill,
            "penalty": _prepare_penalty}[case["op"]](case, g)


def _normal(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _stats_of(v, kind, eps):
    """Mean and reciprocal deviation of each row, from fp64 sums (kind none: 0 and 1)."""
    v = v.double()
    if kind == "none":
        return torch.zeros_like(v[:, 0]), torch.ones_like(v[:, 0])
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    return mean, ((v - mean[:, None]).square().mean(1) + eps).rsqrt()


def _prepare_norm(c, g):
    R, D, res, dt = c["rows"], c["D"], DTYPES[c["res"]], DTYPES[c["dtype"]]
    s = dict(case=c, eps=1e-6)
    for k in ("post", "pre"):
        on = c[k] != "none"
        s[k + "_w"] = _normal(g, D, std=0.2, mean=1.0) if on else None
        s[k + "_b"] = _normal(g, D, std=0.2) if on and c["bias"] and c[k] == "layer" else None
    rpg = c["gate"]
    s["rpg"] = rpg
    s["gate"] = _normal(g, (R + rpg - 1) // rpg, D, std=0.5, mean=0.5, dtype=dt) if rpg else None
    # a residual stream grows with depth: larger than what one block adds
    s["x"] = _normal(g, R, D, std=3.0, mean=0.2, dtype=res)
    s["h"] = _normal(g, R, D, std=0.8, mean=0.1, dtype=dt)
    if c["way"] == "fwd":
        s["out"] = dict(x=torch.empty_like(s["x"]),
                        y=torch.empty(R, D, dtype=dt, device="cuda") if c["pre"] != "none" else None)
    else:
        # the forward's result stands in for x: the backward reads x_out and h
        s["stats"] = torch.stack(_stats_of(s["h"], c["post"], 1e-6) +
                                 _stats_of(s["x"], c["pre"], 1e-6), 1).float()
        s["dx_out"] = _normal(g, R, D, dtype=res)
        s["dy"] = _normal(g, R, D, dtype=dt) if c["pre"] != "none" else None
        vec = lambda k: None if s[k] is None else torch.empty(D, device="cuda")  # noqa: E731
        s["out"] = dict(dx=torch.empty_like(s["x"]), dh=torch.empty_like(s["h"]),
                        dgate=None if not rpg else torch.empty_like(s["gate"]),
                        dpost_w=vec("post_w"), dpost_b=vec("post_b"),
                        dpre_w=vec("pre_w"), dpre_b=vec("pre_b"))
    if own:
        from sparse_gradient_backward_amd import lm
        s["norm"] = lm.BlockNorm(D, post=c["post"], pre=c["pre"], post_weight=s["post_w"],
                                 post_bias=s["post_b"], pre_weight=s["pre_w"],
                                 pre_bias=s["pre_b"], post_eps=1e-6, pre_eps=1e-6,
                                 res_scale=c["scale"])
        s["ws"] = s["norm"].workspace(R) if c["way"] == "bwd" else None
    return s


def _prepare_distill(c, g):
    R, V, K, T = c["rows"], c["V"], c["K"], c["T"]
    # token frequencies: logits fall off with the rank, in an order of their own
    unigram = -torch.log1p(torch.randperm(V, generator=g, device="cuda").float()) * 0.7
    logits = torch.empty(R, V, dtype=DTYPES[c["dtype"]], device="cuda")
    ids = torch.empty(R, K, dtype=torch.int64, device="cuda")
    vals = torch.empty(R, K, device="cuda")
    lse = torch.empty(R, device="cuda")
    for a in range(0, R, 512):
        b = min(R, a + 512)
        logits[a:b] = _normal(g, b - a, V, std=2.0) + unigram
        teacher = logits[a:b].float() + _normal(g, b - a, V, std=0.7)
        vals[a:b], ids[a:b] = teacher.topk(K, dim=1)
        lse[a:b] = torch.logsumexp(teacher.double() / T, 1).float()
    # some rows list fewer entries
    kept = torch.where(torch.rand(R, generator=g, device="cuda") < 0.2,
                       torch.randint(0, K + 1, (R,), generator=g, device="cuda"), K)
    ids[torch.arange(K, device="cuda") >= kept[:, None]] = -1
    labels = torch.randint(0, V, (R,), generator=g, device="cuda")
    labels[torch.rand(R, generator=g, device="cuda") < 0.1] = -1     # no label
    weights = torch.rand(R, generator=g, device="cuda") + 0.5
    weights[torch.rand(R, generator=g, device="cuda") < 0.1] = 0     # padding tokens
    s = dict(case=c, logits=logits, ids=ids, vals=vals, lse=lse if c["tail"] else None,
             labels=labels if c["ce"] else None, weights=weights,
             loss=torch.empty(R, device="cuda"), scale=1.0 / R,
             grad=torch.empty_like(logits) if c["way"] != "loss" else None)
    if c["way"] == "split":
        s["grad_loss"] = torch.rand(R, generator=g, device="cuda") + 0.5
    if own:
        from sparse_gradient_backward_amd import lm
        s["distill"] = lm.TopkDistill(V, K, temperature=T, kd_weight=c["kd"], ce_weight=c["ce"])
        s["ws"] = s["distill"].workspace(R)
        s["stats"] = torch.empty(R, 4, device="cuda") if c["way"] == "split" else None
    return s


def _prepare_penalty(c, g):
    R, V, L = c["rows"], c["V"], c["tokens"]
    rand = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    s = dict(case=c, logits=_normal(g, R, V, std=3.0, dtype=DTYPES[c["dtype"]]))
    # Zipf-like tokens, as in text
    s["tokens"] = (torch.exp(rand(R, L) * math.log(V)) - 1).clamp_(0, V - 1).to(torch.int32)
    s["lens"] = (L * (0.25 + 0.75 * rand(R))).round().clamp_(1, L).to(torch.int32)
    s["lens"][0] = L
    s["prompt"] = (s["lens"] * rand(R)).to(torch.int32)
    s["rep"] = 1.0 + 0.3 * rand(R)
    s["freq"] = 0.2 * rand(R)
    s["pres"] = 0.5 * rand(R)
    s["bias_ids"] = s["bias"] = s["mask"] = s["mask_index"] = None
    if c["biases"]:
        n = c["biases"]
        # distinct in a row: one of each of n equal parts of the vocabulary
        part = torch.arange(n, device="cuda") * V // n
        size = (torch.arange(n, device="cuda") + 1) * V // n - part
        s["bias_ids"] = (part + (rand(R, n) * size).long()).clamp_(max=V - 1).to(torch.int32)
        s["bias_ids"][rand(R, n) < 0.2] = -1
        s["bias"] = _normal(g, R, n, std=4.0)
    if c["masks"]:
        words = (V + 31) // 32
        # half of the states leave a few tokens, the others about half of all
        few = torch.zeros(c["masks"], words, dtype=torch.int32, device="cuda")
        at = rand(c["masks"], words).topk(20, dim=1).indices
        few.scatter_(1, at, (1 << torch.randint(0, 31, at.shape, generator=g, device="cuda")).int())
        half = torch.randint(-2**31, 2**31, few.shape, generator=g, device="cuda").int()
        even = (torch.arange(c["masks"], device="cuda") % 2 == 0)[:, None]
        s["mask"] = torch.where(even, few, half)
        s["mask_index"] = torch.randint(-1, c["masks"], (R,), generator=g, device="cuda").int()
    s["out"] = torch.empty_like(s["logits"])
    if own:
        from sparse_gradient_backward_amd import lm
        s["penalty"] = lm.LogitsPenalty(V)
        s["ws"] = s["penalty"].workspace(R)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op, way = s["case"]["op"], s["case"].get("way")
    if own:
        return _own_norm(s, way) if op == "norm" else \
            _own_distill(s, way) if op == "distill" else _own_penalty(s)
    if op == "norm":
        return _plain_norm_fwd(s) if way == "fwd" else _plain_norm_bwd(s)
    return _plain_distill(s, way) if op == "distill" else _plain_penalty(s)


def _own_norm(s, way):
    o = s["out"]
    if way == "fwd":
        s["norm"].forward(s["x"], s["h"], o["x"], o["y"], gate=s["gate"], rows_per_gate=s["rpg"])
    else:
        s["norm"].backward(s["dx_out"], s["dy"], s["x"], s["h"], s["stats"], o["dx"], o["dh"],
                           gate=s["gate"], rows_per_gate=s["rpg"], d_gate=o["dgate"],
                           d_post_weight=o["dpost_w"], d_post_bias=o["dpost_b"],
                           d_pre_weight=o["dpre_w"], d_pre_bias=o["dpre_b"], workspace=s["ws"])
    return o


def _own_distill(s, way):
    d, args = s["distill"], (s["logits"], s["ids"], s["vals"])
    kw = dict(teacher_lse=s["lse"], labels=s["labels"], row_weights=s["weights"],
              workspace=s["ws"])
    if way == "both":
        d.loss_grad(*args, s["loss"], s["grad"], grad_scale=s["scale"], **kw)
    else:
        d.forward(*args, s["loss"], stats=s["stats"], **kw)
        if way == "split":
            d.backward(*args, s["stats"], s["grad_loss"], s["grad"], grad_scale=s["scale"], **kw)
    return dict(loss=s["loss"], grad=s["grad"])


def _own_penalty(s):
    s["penalty"].apply(s["logits"], s["out"], tokens=s["tokens"], prompt_lens=s["prompt"],
                       lens=s["lens"], repetition=s["rep"], frequency=s["freq"],
                       presence=s["pres"], bias_ids=s["bias_ids"], bias_values=s["bias"],
                       mask=s["mask"], mask_index=s["mask_index"], workspace=s["ws"])
    return s["out"]


def _normed(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v * (v.square().mean(1, keepdim=True) + eps).rsqrt()


def _gate_rows(s):
    """The gate's row of each row, in fp32 (a view where they all share one)."""
    if s["gate"] is None:
        return None
    gate, rows = s["gate"].float(), s["case"]["rows"]
    return gate if s["rpg"] == 1 or gate.shape[0] == 1 else \
        gate.repeat_interleave(s["rpg"], 0)[:rows]


def _plain_norm_fwd(s):
    c = s["case"]
    z = s["h"].float()
    if c["post"] != "none":
        z = _normed(z, c["post"], s["eps"]) * s["post_w"]
        z = z if s["post_b"] is None else z + s["post_b"]
    gate = _gate_rows(s)
    z = z if gate is None else z * gate
    x = z + s["x"].float() * c["scale"]
    y = None
    if c["pre"] != "none":
        y = _normed(x, c["pre"], s["eps"]) * s["pre_w"]
        y = (y if s["pre_b"] is None else y + s["pre_b"]).to(s["h"].dtype)
    return dict(x=x.to(s["x"].dtype), y=y)


def _norm_grad(a, u, rs, kind):
    """Gradient through u = (v - mean) rs of sum(a u)."""
    d = a - u * (a * u).mean(1, keepdim=True)
    return (d - a.mean(1, keepdim=True) if kind == "layer" else d) * rs


def _plain_norm_bwd(s):
    c, st = s["case"], s["stats"]
    o = dict(dgate=None, dpost_w=None, dpost_b=None, dpre_w=None, dpre_b=None)
    t = s["dx_out"].float()
    if c["pre"] != "none":
        dy = s["dy"].float()
        u = (s["x"].float() - st[:, 2:3]) * st[:, 3:4]
        o["dpre_w"] = (dy * u).sum(0)
        o["dpre_b"] = None if s["pre_b"] is None else dy.sum(0)
        t = t + _norm_grad(dy * s["pre_w"], u, st[:, 3:4], c["pre"])
    o["dx"] = (t * c["scale"]).to(s["x"].dtype)
    v = s["h"].float()
    z = v
    if c["post"] != "none":
        v = (v - st[:, 0:1]) * st[:, 1:2]
        z = v * s["post_w"]
        z = z if s["post_b"] is None else z + s["post_b"]
    gate, rpg, R, D = _gate_rows(s), s["rpg"], c["rows"], c["D"]
    if gate is not None:
        dg = t * z
        if rpg > 1:
            G = s["gate"].shape[0]
            full = R // rpg
            parts = [dg[:full * rpg].view(full, rpg, D).sum(1)] if full else []
            dg = torch.cat(parts + ([dg[full * rpg:].sum(0, keepdim=True)] if full < G else []))
        o["dgate"] = dg.to(s["gate"].dtype)
        t = t * gate
    if c["post"] != "none":
        o["dpost_w"] = (t * v).sum(0)
        o["dpost_b"] = None if s["post_b"] is None else t.sum(0)
        t = _norm_grad(t * s["post_w"], v, st[:, 1:2], c["post"])
    o["dh"] = t.to(s["h"].dtype)
    return o


def _plain_distill(s, way):
    c = s["case"]
    V, T = c["V"], c["T"]
    x = s["logits"].float()
    there = s["ids"] >= 0
    at = s["ids"].clamp(min=0)
    off = torch.finfo(torch.float32).min
    # the teacher's distribution over what it lists; with its log-sum-exp, in
    # fp64: what the listed ones leave over is a small difference
    if s["lse"] is None:
        t = torch.where(there, s["vals"] / T, off)
        e = torch.where(there, torch.exp(t - t.max(1, keepdim=True).values), 0)
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total > 0, total, 1)
    else:
        p64 = torch.where(there, torch.exp(s["vals"].double() / T - s["lse"].double()[:, None]), 0)
        p, p_tail = p64.float(), (1 - p64.sum(1, keepdim=True)).clamp(min=0).float()
    top = x.max(1, keepdim=True).values
    e = torch.exp((x - top) / T)
    total = e.sum(1, keepdim=True)
    log_q = ((x.gather(1, at) - top) / T) - total.log()
    kl = torch.where(p > 0, p * (p.clamp(min=1e-38).log() - log_q), 0).sum(1)
    factor = 1.0
    if s["lse"] is not None:
        outside = torch.ones(x.shape[0], V + 1, dtype=torch.bool, device=x.device)
        outside.scatter_(1, torch.where(there, s["ids"], V), False)
        outside = outside[:, :V]
        q_tail = torch.where(outside, e, 0).sum(1, keepdim=True) / total
        kl = kl + torch.where(p_tail > 0, p_tail * (p_tail.clamp(min=1e-38) / q_tail).log(), 0)[:, 0]
        factor = torch.where(outside, 1 - p_tail / q_tail, 1.0)
    some = there.any(1)        # a row that lists nothing has nothing to learn from the teacher
    kl = torch.where(some, kl, 0)
    factor = torch.where(some[:, None], factor, 0.0)
    loss = c["kd"] * T * T * kl
    ce_on = None
    if c["ce"]:
        e1 = e if T == 1 else torch.exp(x - top)
        total1 = e1.sum(1, keepdim=True)
        ce_on = s["labels"] >= 0
        label = s["labels"].clamp(min=0)[:, None]
        ce = total1.log() - (x.gather(1, label) - top)
        loss = loss + c["ce"] * torch.where(ce_on, ce[:, 0], 0)
    loss = loss * s["weights"]
    if way == "loss":
        return dict(loss=loss, grad=None)
    above = s["weights"] * s["scale"]
    above = (above if way == "both" else above * s["grad_loss"])[:, None]
    grad = e / total * factor * (c["kd"] * T)
    grad.scatter_add_(1, at, -p * (c["kd"] * T))
    if c["ce"]:
        w1 = torch.where(ce_on, c["ce"], 0.0)[:, None]
        grad = grad + e1 / total1 * w1
        grad.scatter_add_(1, label, -w1)
    return dict(loss=loss, grad=(grad * above).to(s["logits"].dtype))


def _plain_penalty(s):
    c = s["case"]
    R, V, L = c["rows"], c["V"], c["tokens"]
    x = s["logits"].float()
    place = torch.arange(L, device=x.device)
    said = (place >= s["prompt"][:, None]) & (place < s["lens"][:, None])
    given = place < s["prompt"][:, None]
    tokens = s["tokens"].long()
    count = torch.zeros_like(x).scatter_add_(1, tokens, said.float())
    seen = torch.zeros_like(x).scatter_add_(1, tokens, (said | given).float()) > 0
    rep = s["rep"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][:, None] * count - s["pres"][:, None] * (count > 0)
    if s["bias"] is not None:
        x.scatter_add_(1, s["bias_ids"].clamp(min=0).long(),
                       torch.where(s["bias_ids"] >= 0, s["bias"], 0))
    if s["mask"] is not None:
        j = torch.arange(V, device=x.device)
        bits = ((s["mask"][:, j >> 5] >> (j & 31)) & 1) == 0
        barred = bits[s["mask_index"].clamp(min=0).long()] & (s["mask_index"] >= 0)[:, None]
        x = torch.where(barred, float("-inf"), x)
    return x.to(s["logits"].dtype)


# ------------------------------------------------------------------ work of one pass

def work(case):
    c = case
    if c["op"] == "norm":
        R, D = c["rows"], c["D"]
        res, el = SIZE[c["res"]], SIZE[c["dtype"]]
        pre, gate = c["pre"] != "none", (R + c["gate"] - 1) // c["gate"] * D * el if c["gate"] else 0
        params = 4 * D * ((c["post"] != "none") + pre)
        if c["way"] == "fwd":
            return dict(bytes=R * D * (2 * res + el + el * pre) + gate + params, flops=14 * R * D)
        return dict(bytes=R * D * ((2 + pre) * res + (2 + pre) * el) + 2 * gate + 2 * params + 16 * R,
                    flops=32 * R * D)
    if c["op"] == "distill":
        R, V = c["rows"], c["V"]
        grad = c["way"] != "loss"
        small = R * (12 * c["K"] + 8 + 4 * c["tail"] + 8 * (c["ce"] > 0))
        exps = (1 + (c["ce"] > 0 and c["T"] != 1)) * (1 + grad)
        return dict(bytes=R * V * SIZE[c["dtype"]] * (1 + grad) + small, flops=R * V * exps * 6)
    R, V = c["rows"], c["V"]
    return dict(bytes=2 * R * V * SIZE[c["dtype"]] + R * (4 * c["tokens"] * 5 // 8 + 8 * c["biases"] + 24)
                + c["masks"] * V // 8, flops=4 * R * V)


# ------------------------------------------------------------------ the definitions in fp64

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm_fwd(s) if case["way"] == "fwd" else _exact_norm_bwd(s)
    return _exact_distill(s) if case["op"] == "distill" else _exact_penalty(s)


def _d64(v):
    return None if v is None else v.double()


def _exact_norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    var, mean = torch.var_mean(v, 1, correction=0, keepdim=True)
    u = (v - mean) / torch.sqrt(var + eps) if kind == "layer" else \
        v / torch.sqrt(var + mean * mean + eps)
    return torch.addcmul(0 if b is None else b, u, w) if b is not None else u * w


def _exact_gate(s, gate):
    R = s["case"]["rows"]
    return 1.0 if gate is None else gate[torch.arange(R, device="cuda") // s["rpg"]]


def _exact_norm_fwd(s):
    c = s["case"]
    x = c["scale"] * _d64(s["x"]) + _exact_gate(s, _d64(s["gate"])) * _exact_norm(
        _d64(s["h"]), c["post"], _d64(s["post_w"]), _d64(s["post_b"]), s["eps"])
    y = None if c["pre"] == "none" else _exact_norm(x, c["pre"], _d64(s["pre_w"]),
                                                     _d64(s["pre_b"]), s["eps"])
    return dict(x=x, y=y)


def _exact_norm_bwd(s):
    c = s["case"]
    keys = ("h", "gate", "post_w", "post_b", "pre_w", "pre_b")
    v = {k: None if s[k] is None else s[k].double().requires_grad_() for k in keys}
    x = s["x"].double().requires_grad_()
    t, o = _d64(s["dx_out"]), {}

    def grads(out, above, **leaves):
        at = {k: l for k, l in leaves.items() if l is not None}
        got = torch.autograd.grad(out, list(at.values()), above, materialize_grads=True,
                                  allow_unused=True)
        o.update({k: None for k in leaves})
        o.update(zip(at, got))

    if c["pre"] != "none":
        grads(_exact_norm(x, c["pre"], v["pre_w"], v["pre_b"], s["eps"]), _d64(s["dy"]),
              dx=x, dpre_w=v["pre_w"], dpre_b=v["pre_b"])
        t = t + o["dx"]
    else:
        o.update(dpre_w=None, dpre_b=None)
    z = _exact_gate(s, v["gate"]) * _exact_norm(v["h"], c["post"], v["post_w"], v["post_b"], s["eps"])
    grads(z, t, dh=v["h"], dgate=v["gate"], dpost_w=v["post_w"], dpost_b=v["post_b"])
    o["dx"] = c["scale"] * t
    return o


def _exact_distill(s):
    c = s["case"]
    R, V, T = c["rows"], c["V"], c["T"]
    losses, grads = [], []
    step = max(1, min(R, (1 << 26) // V))
    for a in range(0, R, step):
        r = slice(a, min(R, a + step))
        x = s["logits"][r].double().requires_grad_(c["way"] != "loss")
        ids, there = s["ids"][r], s["ids"][r] >= 0
        t = torch.where(there, s["vals"][r].double() / T, -torch.inf)
        some = there.any(1)
        lse = torch.logsumexp(t, 1) if s["lse"] is None else s["lse"][r].double()
        lse = torch.where(torch.isfinite(lse), lse, 0)
        p = torch.exp(t - lse[:, None])
        log_q = torch.log_softmax(x / T, 1)
        listed_q = log_q.gather(1, ids.clamp(min=0))
        kl = torch.where(p > 0, torch.special.xlogy(p, p) - p * listed_q, 0).sum(1)
        if s["lse"] is not None:
            rest = (1 - p.sum(1)).clamp(min=0)
            gone = torch.zeros(x.shape[0], V + 1, dtype=torch.bool, device=x.device)
            gone.scatter_(1, torch.where(there, ids, V), True)
            log_rest = torch.logsumexp(log_q.masked_fill(gone[:, :V], -torch.inf), 1)
            kl = kl + torch.where(rest > 0, torch.special.xlogy(rest, rest) - rest * log_rest, 0)
        loss = c["kd"] * T ** 2 * torch.where(some, kl, 0)
        if c["ce"]:
            lab = s["labels"][r]
            nll = -torch.log_softmax(x, 1).gather(1, lab.clamp(min=0)[:, None])[:, 0]
            loss = loss + c["ce"] * torch.where(lab >= 0, nll, 0)
        loss = loss * s["weights"][r].double()
        losses.append(loss.detach())
        if c["way"] != "loss":
            above = torch.full_like(loss, s["scale"])
            if c["way"] == "split":
                above = above * s["grad_loss"][r].double()
            grads.append(torch.autograd.grad(loss, x, above)[0])
        del x, log_q
    return dict(loss=torch.cat(losses), grad=torch.cat(grads) if grads else None)


def _exact_penalty(s):
    c = s["case"]
    out = s["logits"].double()
    for r in range(c["rows"]):
        n, m = int(s["prompt"][r]), int(s["lens"][r])
        words = s["tokens"][r].long()
        said = torch.bincount(words[n:m], minlength=c["V"]).double()
        known = (torch.bincount(words[:m], minlength=c["V"]) > 0).nonzero()[:, 0]
        rep = s["rep"][r].double()
        v = out[r]
        v[known] = torch.maximum(v[known], v[known] * 0) / rep + torch.minimum(v[known], v[known] * 0) * rep
        v -= s["freq"][r].double() * said + s["pres"][r].double() * said.sign()
        if s["bias"] is not None:
            on = s["bias_ids"][r] >= 0
            v.index_add_(0, s["bias_ids"][r][on].long(), s["bias"][r][on].double())
        if s["mask"] is not None and int(s["mask_index"][r]) >= 0:
            w = s["mask"][int(s["mask_index"][r])].cpu().numpy().view(np.uint8)
            bits = np.unpackbits(w, bitorder="little")[:c["V"]]
            v[torch.from_numpy(bits == 0).cuda()] = -torch.inf
    return out
