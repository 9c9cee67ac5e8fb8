"""GPU: vocabulary cross-entropy where the label is all but certain: its logit's
gradient is p - 1, the small difference of two numbers near one, and must not be
lost in what a probability is rounded to on the way.

Logits here are exact in fp32 (hidden states are signs, weights few multiples of a
power of two), so that the tolerance holds nothing for them.
"""
import pytest
import torch

import lm_step_reference as ref
from lm_reference import U, half_step
from lm_strict import check
from test_lm_vocab_ce_gpu import make, run

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
V = 300


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def confident(rows, D, dt):
    """Row r has label r and its logit is c, next to those of about e^0.05 of the
    other tokens: 1 - p is some 300 e^-c.  Rows are orthogonal signs, so no label's
    row of the weight adds to another row's logits."""
    s = torch.ones(1, 1)
    while len(s) < D:
        s = torch.cat([torch.cat([s, s], 1), torch.cat([s, -s], 1)])
    g = torch.Generator().manual_seed(0)
    w = torch.randint(-4, 5, (V, D), generator=g).float() / D
    c = torch.tensor([9.0, 10, 11, 12, 13, 14, 15, 30])[torch.arange(rows) % 8]
    w[:rows] = s[:rows] * c[:, None] / D
    return dict(hidden=s[:rows].to(DT[dt]).cuda(), weight=w.to(DT[dt]).cuda(),
                labels=torch.arange(rows).cuda(), row_weights=torch.ones(rows).cuda())


def expected(c, above, dt):
    """A log-sum-exp is off by its own rounding, by those of at most 64 additions
    of parts of a sum of at least one, and by those of the exponentials besides
    the label's: t.  A probability is off by t and its exponential's roundings
    relative to itself, and but for the label's by a half step of fp16 (11 bits,
    subnormals 2^-40) where it waits in that; g then takes one rounding to the
    operands' type."""
    h, w = c["hidden"].double(), c["weight"].double()
    x = h @ w.t()
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    one = torch.zeros_like(p).scatter_(1, c["labels"][:, None], 1.0)
    g = p - one
    said = (x * one).sum(1)
    g[one == 1] = torch.expm1(said - lse)
    reach = 1 + x.amax(1) - x.amin(1)
    t = U * (64 + lse.abs() + 4 * reach * (1 - p.amax(1)))
    wait = 2.0 ** -11 if dt == "bf16" else 0.0
    eg = p * (t[:, None] + U * (8 + 2 * (lse[:, None] - x)) + wait * (1 - one)) + \
        2.0 ** -40 * (1 - one) + (ref.EPS[DT[dt]] + 2 * U) * g.abs()
    dh = above[:, None] * (g @ w)
    tol = above[:, None] * (eg @ w.abs() + ref.chain(V, DT[dt]) * U * (g.abs() @ w.abs()))
    gf, egf = (g * above[:, None]).t(), (eg * above[:, None]).t()
    if dt == "f16":                        # with the factor over the largest
        egf = egf + 2.0 ** -40 * above.max()
    dw = gf @ h
    told = egf @ h.abs() + ref.chain(len(h), DT[dt]) * U * (gf.abs() @ h.abs())
    rest = 1 - p[one == 1]
    assert float(rest.min()) < 1e-10 and 5e-5 < float(rest.sort().values[len(h) // 8]) < 2e-4 \
        and float(rest.max()) > 1e-2
    return {"d_hidden": (dh, half_step(dh, DT[dt]) + tol), "d_weight": (dw, half_step(dw, DT[dt]) + told)}


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,D", [(16, 16), (40, 64), (200, 256)])
@pytest.mark.parametrize("way", ["split", "loss_grad"])
def test_the_gradient_of_a_likely_label(lm, way, rows, D, dt):
    c = confident(rows, D, dt)
    above = torch.rand(rows, device="cuda") + 0.5 if way == "split" else torch.ones(rows, device="cuda")
    o, status = run(lm, c, way, above)
    assert status == "SGB_OK"
    want = expected(c, above.double(), dt)
    check({k: o[k].cpu() for k in want}, {k: (v.cpu(), t.cpu()) for k, (v, t) in want.items()}, way)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,D,tokens", [(3, 1008, 9000), (80, 790, 2880), (128, 512, 5000)])
def test_few_rows_lose_nothing_after_a_forward(lm, rows, D, tokens, dt):
    """As with loss and gradients in one go: gradients of few rows are off by their
    own rounding alone, next to 2^-12 / sqrt(3) of bf16's exponentials."""
    c = make(rows, D, tokens, dt)
    o, _ = run(lm, c, "split")
    want = ref.vocab_ce(c["hidden"], c["weight"], c["labels"], c["row_weights"], None, 1.0, None, DT[dt])
    for k in ("d_hidden", "d_weight"):
        v = want[k][0].double()
        least = (v.to(DT[dt]).double() - v).norm()
        assert float((o[k].double() - v).norm()) <= 1.05 * float(least)
