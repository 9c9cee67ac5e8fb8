"""Vocabulary cross-entropy, dropout and the quantising norm from their
definitions in fp64, and how far an evaluation in fp32 may be from them.

Every function returns {name: (value, tolerance)}: half a step of the output's
type (lm_reference.half_step) plus U = 2^-24 times the roundings on the longest
chain to a value times the magnitudes that enter it.
"""
import numpy as np
import torch

from lm_reference import U, half_step

EPS = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}


def chain(K, dtype):
    """Roundings of a sum of K products: a matrix instruction adds 16 products
    and what there was before (counted as 8 a piece: how it adds them is its
    own), fp32 operands take six products; pieces, parts and a handful of
    factors besides."""
    return (6 if dtype is torch.float32 else 1) * K / 8 + 64


def vocab_ce(hidden, weight, labels, weights=None, above=None, scale=1.0, before=None,
             d_weight_dtype=None):
    """loss, lse, d_hidden, d_weight.

    A logit is off by chain(D) U sum |h w|: `el`.  log-sum-exp: the largest of
    these, and of the exponentials' own roundings (an argument's is relative to
    its size, at most the row's spread of logits; sums of at most 512 terms one
    after another).  A probability is off by these relative to itself, by
    fp16's half step for bf16 operands (where the exponential waits in fp16, of
    subnormals 2^-40), and the gradient of a logit by one rounding to the
    operands' type.
    """
    dt, dev = hidden.dtype, hidden.device
    R, (V, D) = len(hidden), weight.shape
    h, w = hidden.double(), weight.double()
    wt = torch.ones(R, dtype=torch.float64, device=dev) if weights is None else weights.double()
    on = (wt != 0) & (labels >= 0) & (labels < V)
    h = torch.where(on[:, None], h, 0)     # whatever the others hold
    x = h @ w.t()
    el = chain(D, dt) * U * (h.abs() @ w.abs().t())
    lse = torch.logsumexp(x, 1)
    reach = 1 + (x.amax(1) - x.amin(1))
    tl = el.amax(1) + U * (512 + 4 * reach)
    at = labels.clamp(0, V - 1)[:, None]
    said = x.gather(1, at)[:, 0]
    loss = torch.where(on, wt * (lse - said), 0)
    tloss = wt.abs() * (tl + el.gather(1, at)[:, 0] + 4 * U * (lse.abs() + said.abs()))
    out = {"lse": (lse, half_step(lse, torch.float32) + tl),
           "loss": (loss, torch.where(on, half_step(loss, torch.float32) + tloss, 0))}
    f = torch.where(on, wt * (1 if above is None else above.double()), 0)
    p = torch.exp(x - lse[:, None])
    one = torch.zeros_like(p).scatter_(1, at, 1.0)
    g = p - one
    wait = 2.0 ** -11 if dt is torch.bfloat16 else 0
    eg = p * (el + tl[:, None] + U * (8 + 2 * reach[:, None]) + wait) + 2.0 ** -40 + \
        (EPS[dt] + 2 * U) * g.abs()
    if dt is torch.float32:                # three parts of 8 bits, products of them left out
        eg = eg + 2 * U * g.abs()
    del x, el, p, one
    dh = scale * f[:, None] * (g @ w)
    tol = abs(scale) * f.abs()[:, None] * (eg @ w.abs() + chain(V, dt) * U * (g.abs() @ w.abs()))
    out["d_hidden"] = (dh, half_step(dh, dt) + tol)
    gf, egf = (g * f[:, None]).t(), (eg * f.abs()[:, None]).t()
    # with the row's factor over the largest: what fp16 cannot hold of a small one
    egf = egf + (2.0 ** -40 if dt is torch.float16 else 0) * f.abs().max()
    dw = scale * (gf @ h)
    tol = abs(scale) * (egf @ h.abs() + chain(R, dt) * U * (gf.abs() @ h.abs()))
    if before is not None:
        dw = dw + before.double()
        tol = tol + 4 * U * (dw.abs() + before.double().abs())
    out["d_weight"] = (dw, half_step(dw, d_weight_dtype or dt) + tol)
    return out


# ------------------------------------------------------------- dropout

def philox(counter, key):
    """Philox4x32-10 of four arrays of words and two words, in Python's way:
    products of uint64."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = list(key)
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(rows, cols, p, seed, offset, first_row=0):
    r = first_row + np.arange(rows, dtype=np.uint64)[:, None]
    g = np.arange((cols + 7) // 8, dtype=np.uint64)[None]
    z = np.zeros((rows, (cols + 7) // 8), dtype=np.uint64)
    w = philox([g + z, (r & np.uint64(0xFFFFFFFF)) + z, (r >> np.uint64(32)) + z + np.uint64(2**31),
                z + np.uint64(offset & 0xFFFFFFFF)], (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 2)
    bits = bits.reshape(rows, -1)[:, :cols].astype(np.int64)
    return torch.from_numpy(bits >= round(p * 65536))


def dropout(x, p, seed, offset, residual=None, first_row=0, dtype=None):
    """A product or a fused product and sum, after the scale's own rounding: 2 U."""
    cut = round(p * 65536)
    k = kept(*x.shape, p, seed, offset, first_row)
    y = torch.where(k, x.double() * (65536 / (65536 - cut) if cut < 65536 else 0.0), 0)
    mag = y.abs()
    if residual is not None:
        y = y + residual.double()
        mag = mag + residual.double().abs()
    return {"out": (y, torch.where(k, half_step(y, dtype or x.dtype) + 2 * U * mag, 0))}


# ------------------------------------------------------------- quantising norm

MOST = {"int8": 127.0, "fp8": 448.0}


def quant_norm(h, x, weight, eps, form, group):
    """x_out, v and scales.  The squares' sum takes at most 8 + 10 additions, the
    norm a handful of products: N = 40, as a relative error of v (of a v from a
    sum x + h: of the magnitudes of these)."""
    t = h.double() if x is None else h.double() + x.double()
    mag = h.double().abs() + (0 if x is None else x.double().abs())
    rs = 1 / ((t * t).mean(1, keepdim=True) + eps).sqrt()
    w = weight.double()
    v = t * rs * w
    # an error of t moves v, and through the mean of squares all of the row
    tv = 40 * U * (mag * rs * w.abs() + v.abs() * (1 + rs * (mag * mag).mean(1, keepdim=True).sqrt()))
    D, n = h.shape[1], group or h.shape[1]
    scales = torch.stack([v[:, a:a + n].abs().amax(1) for a in range(0, D, n)], 1) / MOST[form]
    ts = torch.stack([tv[:, a:a + n].amax(1) for a in range(0, D, n)], 1) / MOST[form] + 2 * U * scales
    scales = torch.where(scales < 2.0 ** -126, 0, scales)
    return t, mag, v, tv, scales, ts


def check_codes(q, scales, v, tv, form, group, what=""):
    """Every code is the nearest to v / scale, but for what v's error and a
    quotient's rounding leave open; the largest of a group has the largest code."""
    D, n = v.shape[1], group or v.shape[1]
    s = scales.double().repeat_interleave(n, 1)[:, :D]
    c = q.float().double()
    most = MOST[form]
    assert bool((c.abs() <= most).all()), what
    step = torch.ones_like(c)
    if form == "fp8":   # e4m3: three bits after the first, spacing 2^-9 at the least
        step = torch.exp2(torch.floor(torch.log2(c.abs().clamp(min=2.0 ** -6))) - 3)
        # (below a power of two the spacing is half: the larger one holds too)
    far = (c * s - v).abs()
    bad = ~(far <= s * step * 0.5 * (1 + 4 * U) + tv + 4 * U * v.abs()) & (s > 0)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes off, first {bad.nonzero()[0].tolist()}"
    assert bool((c[s == 0] == 0).all()), what
    for a in range(0, D, n):
        there = scales[:, a // n] > 0
        assert bool((c[:, a:a + n].abs().amax(1)[there] == most).all()), what
