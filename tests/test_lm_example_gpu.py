"""GPU: the operators together, as examples/token_model.py uses them: the
training step's gradients against autograd's of the same model in fp64, losses
that fall, and generation that keeps to the grammar and repeats nothing."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "token_model.py")
    spec = importlib.util.spec_from_file_location("token_model", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_loss_falls_and_generation_keeps_to_its_rules(ex):
    m, losses = ex.train(40)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.9 * losses[0], losses
    seq = m.generate(torch.arange(5, device="cuda").int(), 10, ex.even_tokens(m.V)).tolist()
    for s in seq:
        made = s[1:]
        assert all(t % 2 == 0 for t in made) and len(set(made)) == len(made), s


def test_step_against_autograd(ex):
    """One step moves every parameter by lr times the gradient of the mean
    loss: fp32 products of up to 2000 terms, each sum off by at most a rounding
    a term, 2000 * 2^-24 = 1.2e-4 of the magnitudes in it; 2e-3 of the largest
    element leaves room for the magnitudes' ratio to it."""
    m = ex.TokenModel(vocab=600, D=96, hidden=64, rows=80, K=5, seed=3)
    teacher = m.rand(600, 600, std=2.0)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, 50, (80,), generator=g, device="cuda")
    values, ids = teacher[tokens].topk(5, dim=1)
    lse = torch.logsumexp(teacher[tokens].double(), 1).float()
    labels = torch.randint(0, 600, (80,), generator=g, device="cuda")
    names = ("table", "w1", "w2", "head", "gate")
    p = {k: getattr(m, k).double().cpu().requires_grad_() for k in names}
    before = {k: getattr(m, k).clone() for k in names}
    loss = m.step(tokens, labels, ids, values, lse, lr=1.0)

    def rms(v):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
    t, i = tokens.cpu(), ids.cpu()
    x = p["table"][t]
    y = rms(x + p["gate"] * rms(torch.tanh(x @ p["w1"].t()) @ p["w2"].t()))
    lq = torch.log_softmax(y @ p["head"].t(), 1)
    tp = torch.exp(values.double().cpu() - lse.double().cpu()[:, None])
    rest = 1 - tp.sum(1)
    out = torch.ones_like(lq, dtype=torch.bool).scatter_(1, i, False)
    lrest = torch.logsumexp(lq.masked_fill(~out, -torch.inf), 1)
    kl = (tp * (tp.log() - lq.gather(1, i))).sum(1) + rest * (rest.log() - lrest)
    want = (0.7 * kl - 0.3 * lq.gather(1, labels.cpu()[:, None])[:, 0]).mean()
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) < 1e-4 * abs(want)
    for k in names:
        got = (before[k] - getattr(m, k)).double().cpu()
        ref = p[k].grad
        # the difference of two fp32 values is off by a rounding of theirs too
        tol = 2e-3 * ref.abs().max() + 2.0 ** -23 * before[k].abs().max().cpu().double()
        assert float((got - ref).abs().max()) < float(tol), k
