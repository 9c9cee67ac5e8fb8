"""GPU: every token-model call on a stream of its own, and captured into a HIP
graph: replayed with eager work and synchronisations between the replays, each
replay bit-equal to the eager call on the same inputs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def norm_calls(lm):
    R, D = 300, 1000
    g = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, h, gate, dxo, dy = n(R, D), n(R, D).bfloat16(), n(3, D).bfloat16(), n(R, D), n(R, D).bfloat16()
    norm = lm.BlockNorm(D, post_weight=n(D), pre_weight=n(D))
    ws = norm.workspace(R)
    o = dict(xo=torch.empty_like(x), y=torch.empty_like(h), st=torch.empty(R, 4, device="cuda"),
             dx=torch.empty_like(x), dh=torch.empty_like(h), dg=torch.empty_like(gate),
             w1=torch.empty(D, device="cuda"), w2=torch.empty(D, device="cuda"))

    def call():
        norm.forward(x, h, o["xo"], o["y"], gate=gate, rows_per_gate=100, stats=o["st"])
        norm.backward(dxo, dy, o["xo"], h, o["st"], o["dx"], o["dh"], gate=gate, rows_per_gate=100,
                      d_gate=o["dg"], d_post_weight=o["w1"], d_pre_weight=o["w2"], workspace=ws)
    return call, [x, dy], list(o.values())


def distill_calls(lm):
    R, V, K = 40, 9001, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(R, V, generator=g, device="cuda").bfloat16()
    vals, ids = (x.float() + 0.3).topk(K, dim=1)
    lse = torch.logsumexp(x.float() + 0.3, 1)
    d = lm.TopkDistill(V, K)
    ws, st = d.workspace(R), torch.empty(R, 4, device="cuda")
    loss, grad, loss2, grad2 = (torch.empty(R, device="cuda"), torch.empty_like(x),
                                torch.empty(R, device="cuda"), torch.empty_like(x))

    def call():
        d.loss_grad(x, ids, vals, loss, grad, teacher_lse=lse, workspace=ws)
        d.forward(x, ids, vals, loss2, stats=st, teacher_lse=lse, workspace=ws)
        d.backward(x, ids, vals, st, loss, grad2, teacher_lse=lse, workspace=ws)
    return call, [x, vals], [loss, grad, loss2, grad2, st]


def penalty_calls(lm):
    R, V, L = 20, 7001, 300
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(R, V, generator=g, device="cuda").half()
    tok = torch.randint(0, V, (R, L), generator=g, device="cuda").int()
    rep = torch.rand(R, generator=g, device="cuda") + 1
    p = lm.LogitsPenalty(V)
    ws, out = p.workspace(R), torch.empty_like(x)
    return (lambda: p.apply(x, out, tokens=tok, repetition=rep, frequency=rep, workspace=ws)), \
        [x, rep], [out]


@pytest.mark.parametrize("make", [norm_calls, distill_calls, penalty_calls])
def test_streams_and_graphs(lm, make):
    call, inputs, outputs = make(lm)
    print(make.__name__, flush=True)
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
        # other inputs in the same places, an eager call on them, then the replay
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
