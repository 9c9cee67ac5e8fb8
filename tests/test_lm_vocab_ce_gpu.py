"""GPU: vocabulary cross-entropy against its fp64 definition, element by
element: loss alone, loss and gradients in one go, forward then backward."""
import pytest
import torch

import lm_step_reference as ref
from lm_strict import check

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def make(rows, D, V, dt, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    c = dict(hidden=n(rows, D).to(DT[dt]), weight=(n(V, D) * (std / D ** 0.5)).to(DT[dt]),
             labels=torch.randint(0, V, (rows,), generator=g, device="cuda"),
             row_weights=torch.rand(rows, generator=g, device="cuda") + 0.5)
    c["labels"][1::7] = -1
    c["row_weights"][2::5] = 0
    return c


def run(lm, c, way="loss_grad", above=None, scale=1.0, before=None, wt=None, lse_given=True, what=""):
    """The call's outputs and status."""
    rows, D = c["hidden"].shape
    V = len(c["weight"])
    what += f" {way} rows={rows} D={D} V={V} {c['hidden'].dtype}"
    print(what, flush=True)
    dt = c["hidden"].dtype
    p = lm.VocabCrossEntropy(D, V)
    ws = p.workspace(rows, dt, gradient=way != "forward")
    ws.fill_(0x7f)                # what a workspace holds before a call is no number
    o = dict(loss=torch.full((rows,), 9.0, device="cuda"), lse=torch.full((rows,), 9.0, device="cuda"),
             d_hidden=torch.full_like(c["hidden"], 9.0),
             d_weight=torch.full_like(c["weight"], 9.0, dtype=wt or dt) if before is None else before.clone())
    args = (c["hidden"], c["weight"], c["labels"])
    kw = dict(row_weights=c["row_weights"], workspace=ws)
    gr = dict(grad_scale=scale, accumulate=before is not None, d_hidden=o["d_hidden"],
              d_weight=o["d_weight"])
    if way == "forward":
        p.forward(*args, o["loss"], lse=o["lse"], **kw)
        del o["d_hidden"], o["d_weight"]
    elif way == "loss_grad":
        p.loss_grad(*args, o["loss"], lse=o["lse"] if lse_given else None, **gr, **kw)
        if not lse_given:
            del o["lse"]
    else:
        p.forward(*args, o["loss"], lse=o["lse"], **kw)
        assert p.device_status(ws) == "SGB_OK"
        p.backward(*args, o["lse"], above, **gr, **kw)
    return o, p.device_status(ws)


def test(o, c, above=None, scale=1.0, before=None, what=""):
    want = ref.vocab_ce(c["hidden"], c["weight"], c["labels"], c["row_weights"], above, scale, before,
                        o["d_weight"].dtype if "d_weight" in o else None)
    on = c["labels"] >= 0                 # the others have the lse of whatever they hold
    if c["row_weights"] is not None:
        on &= c["row_weights"] != 0
    o = {**o}
    if "lse" in o:
        o["lse"] = torch.where(on, o["lse"], 0)
        want["lse"] = tuple(torch.where(on, t, 0) for t in want["lse"])
    check({k: v.cpu() for k, v in o.items()}, {k: (v.cpu(), t.cpu()) for k, (v, t) in want.items()}, what)


test.__test__ = False
SIZES = [(1, 1, 1), (3, 7, 5), (1, 64, 1000), (64, 64, 64), (65, 72, 257), (130, 129, 1025),
         (257, 200, 300), (300, 320, 4101)]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,D,V", SIZES)
def test_all_ways(lm, rows, D, V, dt):
    c = make(rows, D, V, dt)
    scale = 1.0 if dt == "f16" else 1.0 / rows
    for way in ("forward", "loss_grad"):
        o, status = run(lm, c, way, scale=scale)
        assert status == "SGB_OK"
        test(o, c, scale=scale, what=way)
    above = torch.rand(rows, device="cuda") + 0.5
    o, status = run(lm, c, "split", above=above, scale=scale)
    assert status == "SGB_OK"
    test(o, c, above, scale, what="split")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_large_tiles(lm, dt):
    """More rows and columns than the small tiles are taken for."""
    c = make(3001, 640, 20011, dt)
    o, _ = run(lm, c, scale=0.25)
    test(o, c, scale=0.25)


@pytest.mark.parametrize("dt,rows", [("bf16", 700), ("f16", 300), ("f32", 300)])
def test_chunks_and_pieces(lm, dt, rows):
    """A vocabulary whose exponentials take several chunks of rows, and whose
    copies several pieces."""
    c = make(rows, 64, (1 << 20) + 77, dt)
    o, _ = run(lm, c, scale=1.0, lse_given=False)
    test(o, c, scale=1.0)
    if dt == "bf16":
        before = torch.randn(c["weight"].shape, device="cuda")
        above = torch.rand(rows, device="cuda")
        for b in (before, before.bfloat16()):
            o, _ = run(lm, c, "split", above, scale=1.0, before=b)
            test(o, c, above, 1.0, b)


@pytest.mark.parametrize("V", [1 << 20, (1 << 20) + 77])
@pytest.mark.parametrize("dt,rows", [("bf16", 1100), ("f16", 700), ("f32", 700)])
def test_more_chunks(lm, dt, rows, V):
    """Several chunks of rows with several pieces each, of a weight whose rows are
    read where they are throughout and of one that takes copies."""
    c = make(rows, 64, V, dt)
    o, _ = run(lm, c)
    test(o, c)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 16, 17, 40, 100])
def test_few_rows_of_whole_tiles(lm, rows, dt):
    """Tiles for few rows, of a weight that is read where it is in every product."""
    c = make(rows, 256, 32768, dt)
    for way, above in (("loss_grad", None), ("split", torch.rand(rows, device="cuda") + 0.5)):
        o, _ = run(lm, c, way, above)
        test(o, c, above)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,D,V", [(1030, 64, 20000), (2100, 128, 9000), (500, 1088, 4000)])
def test_short_sums(lm, rows, D, V, dt):
    """Products whose summed dimension is short: few columns, few rows."""
    c = make(rows, D, V, dt)
    o, _ = run(lm, c)
    test(o, c)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,D,V", [(33, 4096, 65600), (7, 16384, 20032)])
def test_large_weight(lm, rows, D, V, dt):
    """A weight of more than a piece's copies hold, whole steps long: it is read
    where it is, and the gradients' pieces are longer than a copy's."""
    c = make(rows, D, V, dt)
    o, _ = run(lm, c)
    test(o, c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_chunks_of_long_rows(lm, dt):
    """So many rows of so many columns that their copies take two chunks."""
    rows, D, V = 8200, 16384, 70
    c = make(rows, D, V, dt)
    p = lm.VocabCrossEntropy(D, V)
    assert p.workspace_bytes(2 * rows, DT[dt]) < p.workspace_bytes(rows, DT[dt]) * 1.01 + 16 * rows
    o, _ = run(lm, c)
    test(o, c)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_large_weight_of_odd_address(lm, dt):
    """A weight that begins at an odd element: its copy takes several pieces."""
    rows, D, V = 33, 4096, 40003
    c = make(rows, D, V, dt)
    wide = torch.full((V, D + 8), float("nan"), dtype=DT[dt], device="cuda")
    wide[:, 1:D + 1] = c["weight"]
    c["weight"] = wide[:, 1:D + 1]
    for way in ("loss_grad", "split"):
        o, _ = run(lm, c, way)
        test(o, c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_far_apart(lm, dt):
    """Rows further apart than 32 bits of bytes reach over a tile."""
    rows, D, V, apart = 40, 64, 300, 1 << 22
    c = make(rows, D, V, dt)
    base, _ = run(lm, c)
    for k, n in (("weight", V), ("hidden", rows)):
        wide = torch.empty(n, apart, dtype=DT[dt], device="cuda")
        wide[:, :D] = c[k]
        o, _ = run(lm, {**c, k: wide[:, :D]})
        test(o, c)
        del wide


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,D,V", [(3, 1008, 9000), (80, 790, 2880), (128, 512, 5000)])
def test_few_rows_lose_nothing(lm, rows, D, V, dt):
    """Gradients of few rows are off by their own rounding alone: of rms 2^-8 / sqrt(12)
    or so, next to 2^-12 / sqrt(3) of bf16's exponentials, 0.4% of it squared in."""
    c = make(rows, D, V, dt)
    o, _ = run(lm, c)
    want = ref.vocab_ce(c["hidden"], c["weight"], c["labels"], c["row_weights"], None, 1.0, None, DT[dt])
    for k in ("d_hidden", "d_weight"):
        v = want[k][0].double().to(o[k].device)
        least = (v.to(DT[dt]).double() - v).norm()
        assert float((o[k].double() - v).norm()) <= 1.05 * float(least)


def test_forward_in_chunks(lm):
    """Loss alone: the sums of exponentials take several chunks of rows."""
    rows, D, V = 2200, 8, (1 << 20) + 3
    c = make(rows, D, V, "bf16")
    o, _ = run(lm, c, "forward")
    for a in range(0, rows, 550):
        part = {k: v if k == "weight" else v[a:a + 550] for k, v in c.items()}
        test({k: v[a:a + 550] for k, v in o.items()}, part)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_few_rows_of_a_long_product(lm, dt):
    """d_hidden's sum over the vocabulary is shared out."""
    c = make(5, 256, 30000, dt)
    o, _ = run(lm, c)
    test(o, c)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_strides_and_alignment(lm, dt):
    """Rows of wider buffers that begin at odd elements, in and out."""
    rows, D, V = 70, 128, 500
    c = make(rows, D, V, dt)
    base, _ = run(lm, c)
    for at, W in ((0, 192), (8, 256), (1, 131), (3, 200)):
        wide = {}
        for k in ("hidden", "weight"):
            b = torch.full((len(c[k]), W), float("nan"), dtype=DT[dt], device="cuda")
            b[:, at:at + D] = c[k]
            wide[k] = b[:, at:at + D]
        p = lm.VocabCrossEntropy(D, V)
        ws = p.workspace(rows, DT[dt])
        outs = {k: torch.full((n, W), 5.0, dtype=DT[dt], device="cuda")
                for k, n in (("d_hidden", rows), ("d_weight", V))}
        loss = torch.empty(rows, device="cuda")
        p.loss_grad(wide["hidden"], wide["weight"], c["labels"], loss, outs["d_hidden"][:, at:at + D],
                    outs["d_weight"][:, at:at + D], row_weights=c["row_weights"], workspace=ws)
        assert torch.equal(loss, base["loss"])
        for k in outs:
            assert torch.equal(outs[k][:, at:at + D], base[k]), (k, at, W)
            assert bool((outs[k][:, :at] == 5).all()) and bool((outs[k][:, at + D:] == 5).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,D,V", [(20, 8, 77), (70, 72, 1013), (5, 136, 20001), (600, 328, 3005)])
def test_weight_rows_of_no_whole_steps(lm, rows, D, V, dt):
    """Rows and a vocabulary that end within a step, the weight read where it is:
    NaN behind each row and behind the last."""
    c = make(rows, D, V, dt)
    b = torch.full((V + 1, D + 24), float("nan"), dtype=DT[dt], device="cuda")
    b[:V, :D] = c["weight"]
    c["weight"] = b[:V, :D]
    above = torch.rand(rows, device="cuda") + 0.5
    base = None
    for w in (c["weight"], c["weight"].contiguous()):
        c["weight"] = w
        o, _ = run(lm, c, "split", above)
        test(o, c, above)
        base = base or o
        assert all(torch.equal(o[k], base[k]) for k in o)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_one_gradient_alone(lm, dt):
    c = make(33, 96, 700, dt)
    base, _ = run(lm, c)
    p = lm.VocabCrossEntropy(96, 700)
    ws, loss = p.workspace(33, DT[dt]), torch.empty(33, device="cuda")
    for k in ("d_hidden", "d_weight"):
        out = torch.empty_like(base[k])
        p.loss_grad(c["hidden"], c["weight"], c["labels"], loss, row_weights=c["row_weights"],
                    workspace=ws, **{k: out})
        assert torch.equal(out, base[k])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_accumulates(lm, dt):
    c = make(40, 72, 600, dt)
    for wt in {DT[dt], torch.float32}:
        before = torch.randn(600, 72, device="cuda").to(wt)
        o, _ = run(lm, c, scale=0.5, before=before)
        test(o, c, scale=0.5, before=before)


def test_fp32_weight_gradient_of_bf16(lm):
    c = make(90, 128, 900, "bf16")
    o, _ = run(lm, c, wt=torch.float32)
    test(o, c)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_rows_that_do_not_count(lm, dt):
    """Padding holds NaN and infinities; nothing of it comes through."""
    c = make(50, 64, 400, dt)
    clean, _ = run(lm, c)
    off = (c["row_weights"] == 0) | (c["labels"] < 0)
    assert 5 < int(off.sum()) < 45
    d = {**c, "hidden": c["hidden"].clone()}
    d["hidden"][off] = torch.nan
    d["hidden"][off.nonzero()[0]] = torch.inf
    o, status = run(lm, d)
    assert status == "SGB_OK"
    for k in ("loss", "d_hidden", "d_weight"):
        assert torch.equal(o[k], clean[k]), k
    assert bool((o["loss"][off] == 0).all()) and bool((o["d_hidden"][off] == 0).all())
    c["row_weights"][:] = 0
    o, _ = run(lm, c)
    assert not bool(o["loss"].any() | o["d_hidden"].any() | o["d_weight"].any())


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_not_finite(lm, dt):
    """A row with a NaN is NaN, and d_weight with it; the other rows are not touched."""
    c = make(20, 64, 300, dt)
    c["labels"].clamp_(min=0)
    c["row_weights"][:] = 1
    clean, _ = run(lm, c)
    for bad in (torch.nan, torch.inf):
        d = {**c, "hidden": c["hidden"].clone()}
        d["hidden"][4, 9] = bad
        o, _ = run(lm, d)
        rest = torch.arange(20, device="cuda") != 4
        assert bool(o["loss"][4].isnan()) and bool(o["d_hidden"][4].isnan().all())
        assert bool(o["d_weight"].isnan().all())
        assert torch.equal(o["loss"][rest], clean["loss"][rest])
        assert torch.equal(o["d_hidden"][rest], clean["d_hidden"][rest])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_barred_tokens_and_rows_without_mass(lm, dt):
    """Logits of -inf: a column of minus infinity under positive hidden states.
    A row of nothing else has no distribution."""
    c = make(6, 64, 200, dt)
    c["labels"][:] = 7
    c["row_weights"][:] = 1
    c["hidden"].abs_()
    c["weight"][50:60] = -torch.inf
    o, _ = run(lm, c, "forward")
    keep = [v for v in range(200) if not 50 <= v < 60]
    test(o, {**c, "weight": c["weight"][keep]})
    c["weight"][:] = -torch.inf
    o, _ = run(lm, c, "loss_grad")
    assert bool(o["loss"].isnan().all()) and bool(o["d_hidden"].isnan().all())
    assert bool((o["lse"] == -torch.inf).all())


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_wide_spread(lm, dt):
    """Logits hundreds apart, large ones of one sign, the label the likeliest or
    the least likely."""
    c = make(40, 64, 500, dt, std=60.0)
    x = c["hidden"].double() @ c["weight"].double().t()
    c["labels"][::2] = x.argmax(1)[::2]
    c["labels"][1::2] = x.argmin(1)[1::2]
    o, _ = run(lm, c)
    test(o, c)


def test_small_and_large_factors(lm):
    """Row weights and gradients from above of very different sizes, fp16."""
    c = make(40, 64, 500, "f16")
    c["row_weights"] = torch.exp2(torch.randint(-20, 10, (40,), device="cuda").float())
    above = torch.exp2(torch.randint(-10, 16, (40,), device="cuda").float())
    o, _ = run(lm, c, "split", above, scale=2.0 ** -20)
    test(o, c, above, 2.0 ** -20)


def test_labels_past_the_vocabulary(lm):
    c = make(30, 64, 300, "bf16")
    d = {**c, "labels": c["labels"].clone()}
    c["labels"][8] = -1
    clean, _ = run(lm, c)
    for bad in (300, 2**40):
        d["labels"][8] = bad
        d["row_weights"][8] = 1.0
        for way in ("forward", "loss_grad"):
            o, status = run(lm, d, way)
            assert status == "SGB_ERR_INDEX_OUT_OF_RANGE"
            for k in o:
                assert torch.equal(o[k], clean[k]), (way, k)


def test_without_weights(lm):
    c = make(30, 64, 300, "bf16")
    c["row_weights"] = None
    o, _ = run(lm, c)
    test(o, c)


def test_a_workspace_of_more_rows(lm):
    c = make(30, 64, 300, "bf16")
    base, _ = run(lm, c)
    p = lm.VocabCrossEntropy(64, 300)
    ws = p.workspace(5000)
    assert p.workspace_bytes(30) <= ws.numel()
    loss, dh, dw = torch.empty(30, device="cuda"), torch.empty_like(c["hidden"]), torch.empty_like(c["weight"])
    p.loss_grad(c["hidden"], c["weight"], c["labels"], loss, dh, dw, row_weights=c["row_weights"],
                workspace=ws)
    assert torch.equal(loss, base["loss"]) and torch.equal(dh, base["d_hidden"]) and \
        torch.equal(dw, base["d_weight"])


def test_no_rows(lm):
    p = lm.VocabCrossEntropy(64, 300)
    ws = p.workspace(0)
    e = torch.empty(0, 64, device="cuda")
    w = torch.randn(300, 64, device="cuda")
    labels, loss = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    p.forward(e, w, labels, loss, workspace=ws)
    for wt in (torch.float32, ):
        dw = torch.ones(300, 64, dtype=wt, device="cuda")
        p.loss_grad(e, w, labels, loss, torch.empty_like(e), dw, accumulate=True, workspace=ws)
        assert bool((dw == 1).all())
        p.loss_grad(e, w, labels, loss, torch.empty_like(e), dw, workspace=ws)
        assert not bool(dw.any())


def test_gradient_against_differences(lm):
    """Directional differences of the fp64 loss at the kernel's own gradient."""
    c = make(12, 40, 90, "f32")
    o, _ = run(lm, c)
    g = torch.Generator(device="cuda").manual_seed(5)
    on = (c["row_weights"] != 0) & (c["labels"] >= 0)

    def loss(h, w):
        x = h @ w.t()
        at = c["labels"].clamp(min=0)[:, None]
        return (torch.where(on, c["row_weights"].double() *
                            (torch.logsumexp(x, 1) - x.gather(1, at)[:, 0]), 0)).sum()
    h, w = c["hidden"].double(), c["weight"].double()
    for k, d in (("d_hidden", h), ("d_weight", w)):
        u = torch.randn(d.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        up = loss(h + e * u, w) if k == "d_hidden" else loss(h, w + e * u)
        down = loss(h - e * u, w) if k == "d_hidden" else loss(h, w - e * u)
        got = float((o[k].double() * u).sum())
        # a central difference's own error: e^2 times third derivatives, 1e-10 here
        assert abs(got - float((up - down) / (2 * e))) < 1e-4 * float(o[k].double().norm() * u.norm()) / 10
