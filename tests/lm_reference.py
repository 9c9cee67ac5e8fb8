"""The token-model operators' definitions in fp64 on the CPU, and how far an
fp32 evaluation rounded once may be from them.

Every function returns {name: (value, tolerance)}.  A tolerance is half a step
of the output's type (torch.finfo(t).eps / 2 relative to the value, half the
smallest subnormal at the bottom) plus N * 2^-24 times the sum of the
magnitudes that enter the value: N counts the fp32 roundings on the longest
chain to it, products and additions of a tree or of a lane's own columns
alike, taken generously (stated at each).
"""
import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def half_step(v, dtype):
    return torch.finfo(dtype).eps / 2 * v.abs() + TINY[dtype]


# ------------------------------------------------------------- block norms

def _norm(v, kind, w, b, eps):
    """Value, and the magnitude of what it is a difference of."""
    if kind == "none":
        return v, v.abs()
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    rs = 1 / ((v - mean).square().mean(1, keepdim=True) + eps).sqrt()
    y = (v - mean) * rs * w
    mag = (v.abs() + mean.abs() + v.abs().mean(1, keepdim=True)) * rs * w.abs()
    if b is not None:
        y, mag = y + b, mag + b.abs()
    return y, mag


def _rows_of(gate, rpg, rows):
    return 1.0 if gate is None else gate[torch.arange(rows) // rpg]


def norm_forward(x, h, gate, rpg, post, pre, pw, pb, qw, qb, eps, scale):
    """x_out, y: N = 64 (a norm is a tree of at most 8 + 10 additions and a
    handful of products, twice)."""
    rt, dt = x.dtype, h.dtype
    x, h, gate = x.double(), h.double(), None if gate is None else gate.double()
    z, zm = _norm(h, post, pw, pb, eps)
    g = _rows_of(gate, rpg, len(x))
    xo = scale * x + g * z
    xm = (scale * x).abs() + (g if gate is None else g.abs()) * zm
    out = {"x_out": (xo, half_step(xo, rt) + 64 * U * xm)}
    if pre != "none":
        y, _ = _norm(xo, pre, qw, qb, eps)
        mean = xo.mean(1, keepdim=True) if pre == "layer" else torch.zeros_like(xo[:, :1])
        rs = 1 / ((xo - mean).square().mean(1, keepdim=True) + eps).sqrt()
        mag = (xm + xm.mean(1, keepdim=True)) * rs * qw.abs() + \
            y.abs() * (1 + rs * xm.square().mean(1, keepdim=True).sqrt())
        out["y"] = (y, half_step(y, dt) + 64 * U * (mag + (0 if qb is None else qb.abs())))
    return out


def stats_of(h, x, post, pre, eps):
    def one(v, kind):
        v = v.double()
        if kind == "none":
            return torch.zeros(len(v)), torch.ones(len(v))
        mean = v.mean(1) if kind == "layer" else torch.zeros(len(v), dtype=torch.float64)
        return mean, 1 / ((v - mean[:, None]).square().mean(1) + eps).sqrt()
    return torch.stack([*one(h, post), *one(x, pre)], 1).float()


def norm_backward(dxo, dy, xo, h, stats, gate, rpg, post, pre, pw, pb, qw, scale):
    """Gradients by the formulas, from the same stats.  N = 64 as in the
    forward, and a sum over rows adds at most one rounding a row."""
    rt, dt = dxo.dtype, h.dtype
    st = stats.double()
    R = len(dxo)
    dxo, xo, h = dxo.double(), xo.double(), h.double()
    dy = None if dy is None else dy.double()
    gate = None if gate is None else gate.double()
    NR = (64 + R) * U
    out = {}
    t, tm = dxo, dxo.abs()
    if pre != "none":
        mx, rx = st[:, 2:3], st[:, 3:4]
        u, um = (xo - mx) * rx, (xo.abs() + mx.abs()) * rx
        a = dy * qw
        m1, m1m = (a * u).mean(1, keepdim=True), (a.abs() * um).mean(1, keepdim=True)
        d, dm = a - u * m1, a.abs() + um * m1m
        if pre == "layer":
            d, dm = d - a.mean(1, keepdim=True), dm + a.abs().mean(1, keepdim=True)
        t, tm = t + rx * d, tm + rx * dm
        out["d_pre_weight"] = ((dy * u).sum(0), NR * (dy.abs() * um).sum(0))
        out["d_pre_bias"] = (dy.sum(0), NR * dy.abs().sum(0))
    out["dx"] = (scale * t, half_step(scale * t, rt) + 64 * U * abs(scale) * tm)
    v, vm = h, h.abs()
    w = torch.ones(h.shape[1], dtype=torch.float64)
    if post != "none":
        mh, rh = st[:, 0:1], st[:, 1:2]
        v, vm, w = (h - mh) * rh, (h.abs() + mh.abs()) * rh, pw
    z = v * w + (0 if pb is None else pb)
    zm = vm * w.abs() + (0 if pb is None else pb.abs())
    g = _rows_of(gate, rpg, R)
    gm = 1.0 if gate is None else g.abs()
    if gate is not None:
        dg, dgm = torch.zeros_like(gate), torch.zeros_like(gate)
        at = torch.arange(R) // rpg
        dg.index_add_(0, at, t * z)
        dgm.index_add_(0, at, tm * zm)
        out["d_gate"] = (dg, half_step(dg, dt) + (64 + min(rpg, R)) * U * dgm)
    b, bm = t * g * w, tm * gm * w.abs()
    if post != "none":
        out["d_post_weight"] = ((t * g * v).sum(0), NR * (tm * gm * vm).sum(0))
        out["d_post_bias"] = ((t * g).sum(0), NR * (tm * gm).sum(0))
        m1, m1m = (b * v).mean(1, keepdim=True), (bm * vm).mean(1, keepdim=True)
        d, dm = b - v * m1, bm + vm * m1m
        if post == "layer":
            d, dm = d - b.mean(1, keepdim=True), dm + bm.mean(1, keepdim=True)
        b, bm = rh * d, rh * dm
    out["dh"] = (b, half_step(b, dt) + 64 * U * bm)
    return out


# ------------------------------------------------------------- distillation

def distill_loss(x, ids, vals, T, kd, ce, lse, labels, weights):
    """Per-row losses, differentiable in x (fp64, loops: small sizes)."""
    losses = []
    for r in range(len(x)):
        if weights is not None and float(weights[r]) == 0:
            losses.append(x.new_zeros(()))
            continue
        V = x.shape[1]
        on = (ids[r] >= 0) & (ids[r] < V)
        loss = x.new_zeros(())
        lq = torch.log_softmax(x[r] / T, 0)
        if bool(on.any()):
            i, t = ids[r][on], vals[r][on].double() / T
            if lse is None:
                p = torch.softmax(t, 0) if bool((t > -torch.inf).any()) else torch.zeros_like(t)
            else:
                p = torch.exp(t - lse[r].double())
            some = p > 0
            kl = (p[some] * (p[some].log() - lq[i[some]])).sum()
            if lse is not None:
                tail = max(0.0, 1.0 - float(p.sum()))
                out = torch.ones(V, dtype=torch.bool)
                out[i] = False
                if tail > 0:
                    kl = kl + tail * (torch.tensor(tail).double().log() -
                                      torch.logsumexp(lq[out], 0))
            loss = loss + kd * T * T * kl
        if labels is not None and 0 <= int(labels[r]) < V:
            loss = loss - ce * torch.log_softmax(x[r], 0)[int(labels[r])]
        losses.append(loss * (1.0 if weights is None else weights[r].double()))
    return torch.stack(losses)


def distill(logits, ids, vals, T, kd, ce, lse=None, labels=None, weights=None, above=None):
    """loss and grad.  N = 256 per exponential sum: a lane adds at most
    V / 2048 groups of 8, then trees; an exponential's argument is off by a
    rounding of (x - m) / T, which `reach` (the spread of the row's
    logits over T, but for those masked by a huge negative number) bounds."""
    x = logits.double().clone().requires_grad_()
    loss = distill_loss(x, ids, vals, T, kd, ce, lse, labels, weights)
    up = torch.ones(len(x)) if above is None else above
    grad, = torch.autograd.grad(loss, x, up.double())
    loss, v = loss.detach(), logits.double()
    fin = torch.where(v.abs() < 1e30, v, torch.nan)
    spread = [(r[~r.isnan()].max() - r[~r.isnan()].min()) if bool((~r.isnan()).any())
              else torch.tensor(0.).double() for r in fin]
    reach = 1 + torch.stack(spread) / min(T, 1.0)
    w = torch.ones(len(x)).double() if weights is None else weights.double()
    ltol = half_step(loss, torch.float32) + \
        256 * U * w.abs() * (kd * T * T + ce) * (1 + reach)
    V = v.shape[1]
    q = torch.softmax(v / T, 1)
    mag = kd * T * q
    if lse is not None:  # the tail's share, spread over what is not listed
        out = torch.ones(len(v), V + 1, dtype=torch.bool)
        out.scatter_(1, torch.where((ids >= 0) & (ids < V), ids, V), False)
        qo = torch.where(out[:, :V], q, 0)
        p = torch.where((ids >= 0) & (ids < V), torch.exp(vals.double() / T - lse.double()[:, None]), 0)
        tail = (1 - p.sum(1, keepdim=True)).clamp(min=0)
        mag = mag + kd * T * torch.nan_to_num(qo / qo.sum(1, keepdim=True)) * tail
    listed = torch.zeros(len(v), V + 1, dtype=torch.float64)
    listed.scatter_(1, torch.where((ids >= 0) & (ids < V), ids, V), 1.0)
    mag = mag + kd * T * listed[:, :V]
    if labels is not None:
        mag = mag + ce * torch.softmax(v, 1)
        at = torch.zeros(len(v), V + 1, dtype=torch.float64)
        at.scatter_(1, torch.where((labels >= 0) & (labels < V), labels, V)[:, None], 1.0)
        mag = mag + ce * at[:, :V]
    k = (up.double() * w).abs()[:, None]
    gtol = half_step(grad, logits.dtype) + 256 * U * k * torch.nan_to_num(mag) * reach[:, None] \
        + 2.0 ** -126
    return {"loss": (loss, ltol), "grad": (grad, gtol)}


# ------------------------------------------------------------- penalties

def penalty(logits, tokens, prompt, lens, rep, freq, pres, bias_ids, bias, mask, mask_index):
    """N = 8: a quotient or product, a fused product and sum, two sums and up
    to a handful of biases."""
    R, V = logits.shape
    out = logits.double().clone()
    mag = out.abs()
    for r in range(R):
        n = int(lens[r]) if lens is not None else (0 if tokens is None else tokens.shape[1])
        m = int(prompt[r]) if prompt is not None else 0
        rp, f, p = (1.0 if a is None else float(a[r]) for a in (rep, freq, pres))
        f, p = (f if freq is not None else 0.0), (p if pres is not None else 0.0)
        counts, seen = {}, set()
        for i in range(n):
            t = int(tokens[r, i])
            if 0 <= t < V:
                seen.add(t)
                if i >= m:
                    counts[t] = counts.get(t, 0) + 1
        for t in seen:
            x = float(out[r, t])
            out[r, t] = x / rp if x > 0 else x * rp
            mag[r, t] = abs(float(out[r, t]))
        for t, c in counts.items():
            out[r, t] -= f * c + p
            mag[r, t] += f * c + abs(p)
        if bias_ids is not None:
            for k in range(bias_ids.shape[1]):
                t = int(bias_ids[r, k])
                if 0 <= t < V:
                    out[r, t] += float(bias[r, k])
                    mag[r, t] += abs(float(bias[r, k]))
        row = -1 if mask is None else (r if mask_index is None else int(mask_index[r]))
        if 0 <= row < (0 if mask is None else len(mask)):
            words = mask[row].to(torch.int64) & 0xFFFFFFFF
            v = torch.arange(V)
            out[r, (words[v // 32] >> (v % 32)) & 1 == 0] = -torch.inf
    tol = half_step(out, logits.dtype) + 8 * U * mag
    # what the type cannot hold rounds to infinity
    out = torch.where(out.abs() > torch.finfo(logits.dtype).max, out.sign() * torch.inf, out)
    return {"out": (out, tol)}


# ------------------------------------------------------------- comparison

def check(got, want, what=""):
    """got: {name: tensor}; every element within its tolerance; infinities and
    NaNs in the same places."""
    for name, g in got.items():
        v, tol = want[name]
        g = g.detach().cpu().double()
        assert g.shape == v.shape, f"{what} {name}: {tuple(g.shape)} for {tuple(v.shape)}"
        assert torch.equal(g.isnan(), v.isnan()), f"{what} {name}: NaNs differ"
        same = (g == v) | v.isnan()
        err = torch.where(same, 0, (g - v).abs())
        bad = ~(err <= tol) & ~same
        if bool(bad.any()):
            at = tuple(int(i) for i in bad.nonzero()[0])
            raise AssertionError(f"{what} {name}: {int(bad.sum())} of {bad.numel()} off, first at "
                                 f"{at}: {float(g[at])!r} for {float(v[at])!r}, tolerance "
                                 f"{float(tol[at]):.3g}")
