"""GPU: vocabulary cross-entropy with exact gradients asked for: off by their own
rounding alone, for any number of rows, chunks and pieces."""
import pytest
import torch

import lm_step_reference as ref
from lm_strict import check
from test_lm_vocab_ce_gpu import make

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def run(lm, c, way="loss_grad", above=None, scale=1.0, before=None, wt=None, exact=True):
    h, w, labels = c["hidden"], c["weight"], c["labels"]
    (rows, D), V = h.shape, len(w)
    print(f"{way} rows={rows} D={D} V={V} {h.dtype} exact={exact}", flush=True)
    p = lm.VocabCrossEntropy(D, V)
    ws = p.workspace(rows, h.dtype, exact=exact)
    ws.fill_(0x7f)
    loss, lse = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    dh = torch.full_like(h, 9.0)
    dw = torch.full_like(w, 9.0, dtype=wt or h.dtype) if before is None else before.clone()
    kw = dict(row_weights=c["row_weights"], workspace=ws)
    gr = dict(grad_scale=scale, accumulate=before is not None, exact=exact, d_hidden=dh, d_weight=dw)
    if way == "loss_grad":
        p.loss_grad(h, w, labels, loss, lse=lse, **gr, **kw)
    else:
        p.forward(h, w, labels, loss, lse=lse, **kw)
        p.backward(h, w, labels, lse, above, **gr, **kw)
    assert p.device_status(ws) == "SGB_OK"
    return dict(loss=loss, d_hidden=dh, d_weight=dw)


def errors(o, c, above=None, scale=1.0, before=None):
    """Each gradient's error over that of rounding the exact one."""
    wt = o["d_weight"].dtype
    want = ref.vocab_ce(c["hidden"], c["weight"], c["labels"], c["row_weights"], above, scale, before, wt)
    check({k: o[k].cpu() for k in o}, {k: (v.cpu(), t.cpu()) for k, (v, t) in want.items()})
    ratios = {}
    for k in ("d_hidden", "d_weight"):
        v = want[k][0].double()
        ratios[k] = float((o[k].double() - v).norm() / (v.to(o[k].dtype).double() - v).norm())
    return ratios


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,D,V", [(129, 512, 5000), (700, 790, 2880), (2000, 256, 9000), (3001, 640, 20011)])
def test_off_by_their_own_rounding(lm, rows, D, V, dt):
    """Next to it: 2^-12 / sqrt(3) of a probability in fp16, against 2^-8 / sqrt(12)
    or so (bf16), 2^-24 times the square root of the sums' lengths against 2^-11 /
    sqrt(12) (fp16): less than 5%."""
    c = make(rows, D, V, dt)
    above = torch.rand(rows, device="cuda") + 0.5
    for way, up in (("loss_grad", None), ("split", above)):
        e = errors(run(lm, c, way, up), c, up)
        assert max(e.values()) <= 1.05, (way, e)
        if way == "loss_grad":   # (fp16's subnormals hide part of what the others lose)
            less = errors(run(lm, c, exact=False), c)
            assert all(e[k] < less[k] for k in e), (e, less)


@pytest.mark.parametrize("dt,rows", [("bf16", 1100), ("f16", 700)])
@pytest.mark.parametrize("V", [1 << 20, (1 << 20) + 77])
def test_chunks_and_pieces(lm, dt, rows, V):
    c = make(rows, 64, V, dt)
    e = errors(run(lm, c), c)
    assert max(e.values()) <= 1.05, e


def test_a_weight_of_odd_address(lm):
    """Its copy takes several pieces."""
    c = make(300, 4096, 40003, "bf16")
    wide = torch.full((40003, 4104), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:4097] = c["weight"]
    c["weight"] = wide[:, 1:4097]
    e = errors(run(lm, c), c)
    assert max(e.values()) <= 1.05, e


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_accumulates_and_fp32(lm, dt):
    c = make(300, 72, 600, dt)
    for wt in (DT[dt], torch.float32):
        before = torch.randn(600, 72, device="cuda").to(wt)
        errors(run(lm, c, scale=0.5, before=before), c, scale=0.5, before=before)
    # in fp32 nothing hides what a gradient's rounding leaves: with it, 16 bits of g at least
    o = run(lm, c, wt=torch.float32)
    want = ref.vocab_ce(c["hidden"], c["weight"], c["labels"], c["row_weights"])["d_weight"][0]
    assert float((o["d_weight"] - want).norm()) <= 2.0 ** -11 * float(want.norm())


@pytest.mark.parametrize("dt,rows", [("bf16", 100), ("f16", 3), ("f32", 300)])
def test_the_same_where_it_changes_nothing(lm, dt, rows):
    """Up to 128 rows, and fp32: the same bits, asked for or not."""
    c = make(rows, 136, 1000, dt)
    a, b = run(lm, c, exact=True), run(lm, c, exact=False)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_rows_that_do_not_count(lm):
    c = make(400, 64, 700, "bf16")
    clean = run(lm, c)
    off = (c["row_weights"] == 0) | (c["labels"] < 0)
    c["hidden"][off] = torch.nan
    o = run(lm, c)
    assert all(torch.equal(o[k], clean[k]) for k in o)


def test_a_workspace_for_exact_gradients_serves_the_others(lm):
    c = make(300, 64, 700, "bf16")
    p = lm.VocabCrossEntropy(64, 700)
    want = run(lm, c, exact=False)
    ws = p.workspace(500, exact=True)
    o = [torch.empty_like(want[k]) for k in ("loss", "d_hidden", "d_weight")]
    p.loss_grad(c["hidden"], c["weight"], c["labels"], *o, row_weights=c["row_weights"], workspace=ws)
    assert all(torch.equal(a, want[k]) for a, k in zip(o, ("loss", "d_hidden", "d_weight")))


def test_captured(lm):
    c = make(300, 128, 3000, "bf16")
    p = lm.VocabCrossEntropy(128, 3000)
    ws = p.workspace(300, exact=True)
    o = [torch.empty(300, device="cuda"), torch.empty_like(c["hidden"]), torch.empty_like(c["weight"])]

    def call():
        p.loss_grad(c["hidden"], c["weight"], c["labels"], *o, row_weights=c["row_weights"], workspace=ws,
                    exact=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for r in range(3):
        c["hidden"].mul_(1.0 + 0.125 * (r % 2))
        call()
        torch.cuda.synchronize()
        eager = [t.clone() for t in o]
        for t in o:
            t.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, eager)), r
