"""GPU: the operators together: a training step and generation as
examples/token_model.py makes them, a tied head whose gradient is added to the
embedding's, streams, HIP graphs."""
import importlib.util
import os

import pytest
import torch

import lm_step_reference as ref
import sparse_gradient_backward_amd as sgb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


@pytest.fixture(scope="module")
def ex(lm):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "token_model.py")
    spec = importlib.util.spec_from_file_location("token_model", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs(ex):
    m, losses = ex.train(3, on_labels=3)
    assert all(x == x for x in losses)
    mask = ex.even_tokens(m.V)
    for codes in (False, True):
        for s in m.generate(torch.arange(5, device="cuda").int(), 6, mask, codes).tolist():
            assert all(t % 2 == 0 for t in s[1:]) and len(set(s[1:])) == 6, s


def test_step_on_labels_against_autograd(ex):
    """One step moves every parameter by lr times the gradient of the mean loss,
    under the mask of the definition.  The tolerance is that of the step with a
    teacher: fp32 products of up to 600 terms, 2e-3 of the largest element."""
    m = ex.TokenModel(vocab=600, D=96, hidden=64, rows=80, K=5, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, 50, (80,), generator=g, device="cuda")
    labels = torch.randint(0, 600, (80,), generator=g, device="cuda")
    labels[7] = -1
    names = ("table", "w1", "w2", "head", "gate")
    p = {k: getattr(m, k).double().cpu().requires_grad_() for k in names}
    before = {k: getattr(m, k).clone() for k in names}
    loss = m.step_on_labels(tokens, labels, lr=1.0, step=9, seed=77)

    def rms(v):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
    cut = round(0.1 * 65536)
    kept = ref.kept(80, 96, 0.1, 77, 9) * (65536 / (65536 - cut))
    x = p["table"][tokens.cpu()] * kept
    y = rms(x + p["gate"] * rms(torch.tanh(x @ p["w1"].t()) @ p["w2"].t()))
    lq = torch.log_softmax(y @ p["head"].t(), 1)
    on = labels.cpu() >= 0
    want = -(lq.gather(1, labels.cpu().clamp(min=0)[:, None])[:, 0] * on).mean()
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 1e-4 * abs(float(want.detach()))
    for k in names:
        got = (before[k] - getattr(m, k)).double().cpu()
        g64 = p[k].grad
        tol = 2e-3 * g64.abs().max() + 2.0 ** -23 * before[k].abs().max().cpu().double()
        assert float((got - g64).abs().max()) < float(tol), k


def test_tied_head(lm):
    """One table for the embedding and the head: the head's gradient is written,
    the embedding's added to it by sgb's dense backward."""
    V, D, R = 500, 64, 48
    g = torch.Generator(device="cuda").manual_seed(0)
    table = torch.randn(V, D, generator=g, device="cuda") / 4
    tokens = torch.randint(0, 60, (R,), generator=g, device="cuda")
    labels = torch.randint(0, V, (R,), generator=g, device="cuda")
    plan = sgb.Plan([0, V], [0, D], "none")
    ws = plan.workspace(R, 0)
    x = torch.empty(R, D, device="cuda")
    plan.forward(tokens, None, 0, None, table, x, ws)
    drop, head = lm.Dropout(0.2), lm.VocabCrossEntropy(D, V)
    y, dx, loss = torch.empty_like(x), torch.empty_like(x), torch.empty(R, device="cuda")
    drop.forward(x, y, 3)
    grad = torch.full_like(table, 9.0)
    head.loss_grad(y, table, labels, loss, dx, grad, workspace=head.workspace(R, torch.float32))
    drop.backward(dx, dx, 3)
    plan.backward(dx, tokens, None, 0, None, "dense", grad=grad, accumulate=True, workspace=ws)
    t = table.double().cpu().requires_grad_()
    kept = ref.kept(R, D, 0.2, 3, 0) * (65536 / (65536 - round(0.2 * 65536)))
    e = t[tokens.cpu()] * kept
    lq = torch.log_softmax(e @ t.t(), 1)
    want = -lq.gather(1, labels.cpu()[:, None])[:, 0]
    want.sum().backward()
    # fp32 sums of at most 500 terms in six products each, 6 * 500 / 8 + 64 roundings of
    # magnitudes that add up to at most (48 rows) x (2: a probability, one) x max |x|
    tol = 512 * 2.0 ** -24 * 2 * R * float(e.detach().abs().max())
    assert float((grad.cpu().double() - t.grad).abs().max()) < tol
    assert float((loss.cpu().double() - want.detach()).abs().max()) < 512 * 2.0 ** -24 * 16


def head_calls(lm, dt, rows=70, D=96, V=900):
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(rows, D, generator=g, device="cuda").to(dt)
    w = (torch.randn(V, D, generator=g, device="cuda") / 5).to(dt)
    labels = torch.randint(0, V, (rows,), generator=g, device="cuda")
    p = lm.VocabCrossEntropy(D, V)
    ws = p.workspace(rows, dt)
    f = lambda: torch.empty(rows, device="cuda")  # noqa: E731
    o = [f(), f(), torch.empty_like(h), torch.empty_like(w), f(), torch.empty_like(h),
         torch.empty_like(w)]

    def call():
        p.forward(h, w, labels, o[0], lse=o[1], workspace=ws)
        p.backward(h, w, labels, o[1], o[0], o[2], o[3], workspace=ws)
        p.loss_grad(h, w, labels, o[4], o[5], o[6], workspace=ws)
    return call, [h, w], o


def drop_calls(lm):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(50, 300, generator=g, device="cuda").bfloat16()
    res = torch.randn(50, 300, generator=g, device="cuda")
    state = torch.tensor([5, 0], device="cuda")
    d, out, dx = lm.Dropout(0.3), torch.empty_like(res), torch.empty_like(x)

    def call():
        d.forward(x, out, offset=2, residual=res, state=state)
        d.backward(x, dx, offset=2, state=state)
    return call, [x, res], [out, dx]


def quant_calls(lm):
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(50, 1000, generator=g, device="cuda").half()
    x = torch.randn(50, 1000, generator=g, device="cuda").half()
    n = lm.QuantNorm(1000, weight=torch.ones(1000, device="cuda"), form="fp8", group=128)
    q = torch.empty(50, 1000, device="cuda").to(torch.float8_e4m3fn)
    s, xo = torch.empty(50, 8, device="cuda"), torch.empty_like(x)
    return (lambda: n.forward(h, q, s, x=x, x_out=xo)), [h, x], [q.view(torch.uint8), s, xo]


MAKE = {"bf16": lambda lm: head_calls(lm, torch.bfloat16), "f16": lambda lm: head_calls(lm, torch.half),
        "f32": lambda lm: head_calls(lm, torch.float32), "drop": drop_calls, "quant": quant_calls,
        "large": lambda lm: head_calls(lm, torch.bfloat16, 2100, 512, 9000)}


@pytest.mark.parametrize("which", MAKE)
def test_streams_and_graphs(lm, which):
    """On a stream of its own, and captured: each replay bit-equal to the eager
    call on the same inputs, with eager work and synchronisations between."""
    call, inputs, outputs = MAKE[which](lm)
    print(which, flush=True)
    call()
    torch.cuda.synchronize()
    eager = [o.clone() for o in outputs]
    side = torch.cuda.Stream()
    for o in outputs:
        o.fill_(9)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for o, e in zip(outputs, eager):
        assert torch.equal(o, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for r in range(4):
        for t in inputs:
            t.mul_(1.0 + 0.125 * (r % 2))
        call()
        torch.cuda.synchronize()
        eager = [o.clone() for o in outputs]
        for o in outputs:
            o.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        other = torch.arange(1 << 16, device="cuda", dtype=torch.float32).mul_(0.5)
        torch.cuda.synchronize()
        assert float(other[2]) == 1.0
        for o, e in zip(outputs, eager):
            assert torch.equal(o, e), f"replay {r}"


def test_a_replay_draws_new_masks(lm):
    """The seed and step on the device: a captured dropout follows them."""
    x, out = torch.ones(40, 200, device="cuda"), torch.empty(40, 200, device="cuda")
    state = torch.tensor([11, 0], device="cuda")
    d = lm.Dropout(0.5)
    d.forward(x, out, state=state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.forward(x, out, state=state)
        state[1:].add_(1)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal((out != 0).cpu(), ref.kept(40, 200, 0.5, 11, step)), step


def test_two_calls_at_once(lm):
    """On two streams with a workspace each."""
    a, b = head_calls(lm, torch.bfloat16), head_calls(lm, torch.bfloat16)
    b[1][0].mul_(0.5)
    want = []
    for call, _, outs in (a, b):
        call()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, (call, _, _) in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    for (_, _, outs), w in zip((a, b), want):
        for o, e in zip(outs, w):
            assert torch.equal(o, e)
