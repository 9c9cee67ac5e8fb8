"""GPU: distillation where a distribution has no mass: every id listed under the
teacher's true log-sum-exp, rows of nothing but -inf, masked logits outside what
is listed."""
import pytest
import torch

import lm_strict as strict
from lm_reference import U, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def calls(lm, x, ids, vals, lse, labels, T, kd, ce):
    """(loss, grad) of loss_grad, and of forward and then backward."""
    rows, V = x.shape
    d = lm.TopkDistill(V, ids.shape[1], temperature=T, kd_weight=kd, ce_weight=ce)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = (cu(x), cu(ids), cu(vals))
    kw = dict(teacher_lse=cu(lse), labels=cu(labels) if ce else None, workspace=d.workspace(rows))
    out = []
    for _ in range(2):
        out.append((torch.full((rows,), 7.0, device="cuda"), torch.full_like(args[0], 7.0)))
    d.loss_grad(*args, *out[0], **kw)
    stats = torch.empty(rows, 4, device="cuda")
    d.forward(*args, out[1][0], stats=stats, **kw)
    d.backward(*args, stats, None, out[1][1], **kw)
    return out


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K", [(1, 1), (5, 8), (40, 40), (1000, 1024)])
@pytest.mark.parametrize("T,ce", [(1.0, 0.0), (2.0, 0.3), (1.0, 0.3)])
def test_all_listed_and_the_true_log_sum_exp(lm, V, K, dt, T, ce):
    """What 1 - sum p leaves is the rounding of an fp32 log-sum-exp; nothing
    lies outside the listed ids for it to be compared with.  Tolerances: 256
    fp32 roundings of the magnitudes, with exponents off by roundings of
    their arguments, as for any distillation."""
    rows, kd = 64, 0.7
    g = torch.Generator().manual_seed(V)
    x = (2 * torch.randn(rows, V, generator=g)).to(dt)
    teacher = torch.randn(rows, V, generator=g)
    ids = torch.full((rows, K), -1)
    ids[:, :V] = torch.stack([torch.randperm(V, generator=g) for _ in range(rows)])
    vals = torch.zeros(rows, K)
    vals[:, :V] = teacher.gather(1, ids[:, :V])
    lse = torch.logsumexp(teacher.double() / T, 1).float()
    labels = torch.randint(0, V, (rows,), generator=g)
    x64 = x.double().requires_grad_()
    p = torch.exp(teacher.double() / T - lse.double()[:, None])
    loss = kd * T * T * (p * (p.log() - torch.log_softmax(x64 / T, 1))).sum(1)
    if ce:
        loss = loss - ce * torch.log_softmax(x64, 1).gather(1, labels[:, None])[:, 0]
    grad, = torch.autograd.grad(loss.sum(), x64)
    loss = loss.detach()
    reach = 1 + (x.double().amax(1) - x.double().amin(1)) / min(T, 1.0)
    want = {"loss": (loss, half_step(loss, torch.float32) + 256 * U * (kd * T * T + ce) * (1 + reach)),
            "grad": (grad, half_step(grad, dt) + 256 * U * 2 * (kd * T + ce) * reach[:, None])}
    for l, gr in calls(lm, x, ids, vals, lse, labels, T, kd, ce):
        strict.check({"loss": l, "grad": gr}, want, f"V={V} K={K} {dt} T={T} ce={ce}")


@pytest.mark.parametrize("V,rows", [(300, 6), (20011, 6), (20011, 140)])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,ce", [(1.0, 0.0), (2.0, 0.3), (1.0, 0.3)])
def test_rows_of_nothing_but_minus_infinity(lm, V, rows, tail, T, ce):
    """No distribution: loss and gradient are NaN, whatever is listed; the other
    rows' are not."""
    g = torch.Generator().manual_seed(V + rows)
    x = torch.randn(rows, V, generator=g)
    teacher = x + torch.randn(rows, V, generator=g)
    vals, ids = teacher.topk(9, dim=1)
    lse = torch.logsumexp(teacher.double() / T, 1).float() if tail else None
    labels = torch.randint(0, V, (rows,), generator=g)
    x[1] = x[2] = x[4] = -torch.inf
    ids[2] = ids[3] = -1                # nothing listed: with and without a mass
    labels[4] = labels[3] = -1
    none = torch.zeros(rows, dtype=torch.bool)
    none[[1, 2, 4]] = True
    for l, gr in calls(lm, x, ids, vals, lse, labels, T, 0.7, ce):
        assert torch.equal(l.cpu().isnan(), none)
        assert torch.equal(gr.cpu().isnan(), none[:, None].expand(rows, V))
        assert float(l[3]) == 0 and not bool(gr[3].any())


@pytest.mark.parametrize("V", [300, 20011])
def test_a_real_tail_over_masked_logits_is_infinite(lm, V):
    """The teacher gives mass to what the student bars: the divergence is infinite."""
    x = torch.randn(3, V, generator=torch.Generator().manual_seed(1))
    teacher = x.clone()
    vals, ids = teacher.topk(9, dim=1)
    lse = torch.logsumexp(teacher.double(), 1).float()
    x[1] = torch.full((V,), -torch.inf).scatter_(0, ids[1], x[1, ids[1]])
    for l, gr in calls(lm, x, ids, vals, lse, None, 1.0, 1.0, 0.0):
        assert float(l[1]) == torch.inf and bool(l[[0, 2]].isfinite().all())
        assert bool(gr.isfinite().all())


@pytest.mark.parametrize("V,rows", [(300, 64), (20011, 64), (20011, 140)])
@pytest.mark.parametrize("bar", ["-inf", "lowest"])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_logits_barred_for_teacher_and_student(lm, V, rows, bar, T):
    """The listed ids are all that is allowed and the log-sum-exp is theirs: the
    rounding of it is no tail.  Tolerances as above; the gradient of what is
    barred is 0."""
    g = torch.Generator().manual_seed(V)
    K = 9
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(rows)])
    vals, some = torch.randn(rows, K, generator=g), 2 * torch.randn(rows, K, generator=g)
    lse = torch.logsumexp(vals.double() / T, 1).float()
    off = -torch.inf if bar == "-inf" else torch.finfo(torch.float32).min
    x = torch.full((rows, V), off).scatter_(1, ids, some)
    s64 = some.double().requires_grad_()
    p = torch.exp(vals.double() / T - lse.double()[:, None])
    loss = T * T * (p * (p.log() - torch.log_softmax(s64 / T, 1))).sum(1)
    grad, = torch.autograd.grad(loss.sum(), s64)
    loss = loss.detach()
    reach = 1 + some.double().amax(1) - some.double().amin(1)
    for l, gr in calls(lm, x, ids, vals, lse, None, T, 1.0, 0.0):
        strict.check({"loss": l}, {"loss": (loss, half_step(loss, torch.float32) +
                                            256 * U * T * T * (1 + reach))}, f"{V} {rows} {bar}")
        at = gr.gather(1, ids.cuda())
        strict.check({"grad": at}, {"grad": (grad, half_step(grad, torch.float32) +
                                             256 * U * 2 * T * reach[:, None])}, f"{V} {rows} {bar}")
        assert not bool(gr.scatter(1, ids.cuda(), 0.0).any())


def test_a_real_tail_over_the_lowest_value_stays_huge(lm):
    """A tail of the teacher's against q' = exp(-3e38)."""
    V = 300
    x = torch.full((2, V), torch.finfo(torch.float32).min)
    x[:, :5] = 0.0
    ids, vals = torch.arange(5).expand(2, 5).contiguous(), torch.zeros(2, 5)
    p = torch.tensor([0.9, 0.999])                      # listed in all
    lse = (torch.log(torch.tensor(5.0)) - p.log())
    for l, _ in calls(lm, x, ids, vals, lse, None, 1.0, 1.0, 0.0):
        want = (1 - p) * 3.4028235e38
        assert torch.allclose(l.cpu().double(), want.double(), rtol=1e-3)
