"""GPU: distillation from top logits against its fp64 definition and gradient
(by differentiation), element by element: vocabularies either side of the
kernel's steps and splits, K from one up, unlisted and repeated entries, masked
logits, padding rows, out-of-range ids."""
import pytest
import torch

import lm_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def make(rows, V, K, dt, T, tail, ce, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(rows, V, generator=g)).to(DT[dt])
    teacher = x.float() + 0.7 * torch.randn(rows, V, generator=g)
    k = min(K, V)
    vals, ids = torch.zeros(rows, K), torch.full((rows, K), -1)
    vals[:, :k], ids[:, :k] = teacher.topk(k, dim=1)
    if K > 2:
        ids[0, K // 2:] = -1
    lse = torch.logsumexp(teacher.double() / T, 1).float() if tail else None
    labels = torch.randint(0, V, (rows,), generator=g) if ce else None
    if ce and rows > 2:
        labels[1] = -1
        labels[2] = ids[2, 0]          # a label that is listed
    w = torch.rand(rows, generator=g) + 0.5
    return dict(x=x, ids=ids, vals=vals, lse=lse, labels=labels, w=w)


def run(lm, c, T, kd, ce, what=""):
    x = c["x"]
    rows, V = x.shape
    K = c["ids"].shape[1]
    what = f"{what} rows={rows} V={V} K={K} {x.dtype} T={T} kd={kd} ce={ce} tail={c['lse'] is not None}"
    print(what, flush=True)
    d = lm.TopkDistill(V, K, temperature=T, kd_weight=kd, ce_weight=ce)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = (cu(x), cu(c["ids"]), cu(c["vals"]))
    ws = d.workspace(rows)
    kw = dict(teacher_lse=cu(c["lse"]), labels=cu(c["labels"]), row_weights=cu(c["w"]), workspace=ws)
    above = torch.rand(rows, generator=torch.Generator().manual_seed(5)) + 0.5
    scale = 0.25
    want = ref.distill(x, c["ids"], c["vals"], T, kd, ce, c["lse"], c["labels"], c["w"],
                       torch.full((rows,), scale))
    loss, grad = torch.full((rows,), 7.0, device="cuda"), torch.full_like(args[0], 7.0)
    d.loss_grad(*args, loss, grad, grad_scale=scale, **kw)
    ref.check(dict(loss=loss, grad=grad), want, what)
    status = d.device_status(ws)
    loss2, stats = torch.full((rows,), 7.0, device="cuda"), torch.empty(rows, 4, device="cuda")
    d.forward(*args, loss2, stats=stats, **kw)
    ref.check(dict(loss=loss2), want, what + " forward")
    grad2 = torch.full_like(grad, 7.0)
    d.backward(*args, stats, above.cuda(), grad2, grad_scale=scale, **kw)
    want = ref.distill(x, c["ids"], c["vals"], T, kd, ce, c["lse"], c["labels"], c["w"],
                       scale * above)
    ref.check(dict(grad=grad2), want, what + " backward")
    return status


MODES = [(1.0, 1.0, 0.0), (2.0, 0.7, 0.3), (1.0, 0.5, 0.5), (0.7, 0.0, 1.0)]


@pytest.mark.parametrize("V", [1, 5, 8, 31, 2047, 2048, 2049, 5003, 16391])
@pytest.mark.parametrize("tail", [False, True])
def test_vocabularies(lm, V, tail):
    for i, (T, kd, ce) in enumerate(MODES):
        dt = ("f32", "bf16", "f16")[(i + V) % 3]
        c = make(4, V, min(8, V), dt, T, tail, ce)
        if V <= 8 and tail:     # all listed: the teacher leaves nothing for a tail
            t = torch.where(c["ids"] >= 0, c["vals"].double() / T, -torch.inf)
            c["lse"] = torch.logsumexp(t, 1).float() - 1e-3
        run(lm, c, T, kd, ce)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K", [1, 2, 63, 64, 65, 200, 1024])
@pytest.mark.parametrize("tail", [False, True])
def test_listed_counts(lm, dt, K, tail):
    for T, kd, ce in MODES[:3]:
        run(lm, make(5, 3001, K, dt, T, tail, ce, seed=K), T, kd, ce)


@pytest.mark.parametrize("rows,V", [(700, 600), (300, 4100), (1100, 257)])
def test_many_rows(lm, rows, V):
    # one workgroup a row and several
    run(lm, make(rows, V, 16, "bf16", 1.5, True, 0.3), 1.5, 0.7, 0.3)


@pytest.mark.parametrize("tail", [False, True])
def test_longest_rows(lm, tail):
    # past what one workgroup's bits cover: at least two a row whatever the rows
    run(lm, make(2, 140001, 64, "bf16", 1.0, tail, 0.3), 1.0, 0.7, 0.3)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,kd,ce", MODES[:3])
def test_masked_logits(lm, tail, T, kd, ce):
    """-inf and the type's lowest value among the logits, outside and inside
    what is listed; entries with -inf teacher logits; a row with nothing listed."""
    c = make(6, 3000, 12, "bf16", T, tail, ce)
    x = c["x"]
    keep = torch.zeros(3000, dtype=torch.bool)
    keep[c["ids"][3]] = True
    if ce and int(c["labels"][3]) >= 0:
        keep[c["labels"][3]] = True
    x[3, 100:2900] = torch.where(keep[100:2900], x[3, 100:2900], -torch.inf)
    x[4, ::2] = torch.where(torch.zeros(1500).bool() | (c["ids"][4][:, None] ==
                            torch.arange(0, 3000, 2)).any(0), x[4, ::2], torch.finfo(x.dtype).min)
    if ce and int(c["labels"][4]) >= 0:
        x[4, int(c["labels"][4])] = 1.0
    c["vals"][5, 3:6] = -torch.inf
    c["ids"][1] = -1
    run(lm, c, T, kd, ce, "masked")


def test_rows_of_one_value(lm):
    """A row of the type's lowest value is a uniform row."""
    c = make(3, 2500, 4, "f32", 1.0, False, 0.5)
    c["x"][0] = torch.finfo(torch.float32).min
    c["x"][1] = 0
    run(lm, c, 1.0, 0.5, 0.5, "uniform")


def test_all_of_a_vocabulary_listed(lm):
    """No student mass outside the listed ids and none of the teacher's."""
    c = make(4, 40, 40, "f32", 1.0, False, 0.3)
    c["ids"][0] = torch.arange(40)
    teacher = torch.zeros(4, 40).scatter_(1, c["ids"].clamp(min=0), c["vals"])
    c["lse"] = torch.logsumexp(teacher.double(), 1).float() - 1e-3
    run(lm, c, 1.0, 0.7, 0.3, "all listed")


@pytest.mark.parametrize("tail", [False, True])
def test_repeated_ids(lm, tail):
    c = make(4, 900, 20, "f32", 1.0, tail, 0.3)
    c["ids"][1, 5] = c["ids"][1, 2]
    c["ids"][3, 1:4] = c["ids"][3, 0]
    if tail:
        c["lse"] += 0.7
    run(lm, c, 1.0, 0.7, 0.3, "repeated")


def test_padding_rows_are_not_read(lm):
    c = make(5, 2100, 8, "bf16", 1.0, True, 0.3)
    c["w"][0] = 0
    c["w"][3] = 0
    c["x"][3] = torch.nan
    c["lse"][3] = torch.nan
    x = c["x"].clone()
    d = lm.TopkDistill(2100, 8, kd_weight=0.7, ce_weight=0.3)
    loss, grad = torch.full((5,), 7.0, device="cuda"), torch.full((5, 2100), 7.0, device="cuda").bfloat16()
    d.loss_grad(x.cuda(), c["ids"].cuda(), c["vals"].cuda(), loss, grad, teacher_lse=c["lse"].cuda(),
                labels=c["labels"].cuda(), row_weights=c["w"].cuda(), workspace=d.workspace(5))
    assert loss[[0, 3]].tolist() == [0, 0] and not bool(grad[[0, 3]].any())
    assert bool(loss[[1, 2, 4]].isfinite().all())


def test_a_row_without_finite_logits_is_nan(lm):
    c = make(3, 2100, 8, "f32", 1.0, False, 0.0)
    c["x"][1] = -torch.inf
    d = lm.TopkDistill(2100, 8)
    loss, grad = torch.empty(3, device="cuda"), torch.empty(3, 2100, device="cuda")
    d.loss_grad(c["x"].cuda(), c["ids"].cuda(), c["vals"].cuda(), loss, grad,
                workspace=d.workspace(3))
    assert loss.isnan().tolist() == [False, True, False]
    assert bool(grad[1].isnan().all()) and bool(grad[[0, 2]].isfinite().all())


def test_out_of_range_ids_are_left_out_and_reported(lm):
    c = make(4, 700, 6, "f32", 1.0, False, 0.3)
    clean = run(lm, c, 1.0, 0.7, 0.3, "clean")
    assert clean == "SGB_OK"
    c["ids"][1, 2] = 700
    c["ids"][2, 0] = 2**40
    assert run(lm, c, 1.0, 0.7, 0.3, "bad ids") == "SGB_ERR_INDEX_OUT_OF_RANGE"
    c = make(4, 700, 6, "f32", 1.0, False, 0.3)
    c["labels"][0] = 700
    assert run(lm, c, 1.0, 0.7, 0.3, "bad label") == "SGB_ERR_INDEX_OUT_OF_RANGE"


def test_strides(lm):
    rows, V, K = 5, 1003, 7
    c = make(rows, V, K, "f16", 1.0, True, 0.0)
    d = lm.TopkDistill(V, K)
    cu = {k: None if v is None else v.cuda() for k, v in c.items()}
    loss, grad = torch.empty(rows, device="cuda"), torch.empty(rows, V, device="cuda").half()
    kw = dict(teacher_lse=cu["lse"], row_weights=cu["w"], workspace=d.workspace(rows))
    d.loss_grad(cu["x"], cu["ids"], cu["vals"], loss, grad, **kw)

    def wide(t, at, W):
        w = torch.full((rows, W), 3, dtype=t.dtype, device="cuda")
        w[:, at:at + t.shape[1]] = t
        return w, w[:, at:at + t.shape[1]]
    _, x = wide(cu["x"], 1, 1100)
    _, ids = wide(cu["ids"], 2, 11)
    _, vals = wide(cu["vals"], 3, 13)
    wg, g = wide(torch.zeros_like(grad), 5, 1021)
    loss2 = torch.empty_like(loss)
    d.loss_grad(x, ids, vals, loss2, g, **kw)
    assert torch.equal(loss, loss2) and torch.equal(grad, g)
    assert bool((wg[:, :5] == 3).all()) and bool((wg[:, 5 + V:] == 3).all())


def test_differences(lm):
    """grad against differences of the loss (fp32) along it: off by e^2 times
    third derivatives and the loss's rounding over e, both below 1e-2 of it."""
    c = make(3, 400, 6, "f32", 2.0, True, 0.3)
    d = lm.TopkDistill(400, 6, temperature=2.0, kd_weight=0.7, ce_weight=0.3)
    cu = {k: None if v is None else v.cuda() for k, v in c.items()}
    ws = d.workspace(3)
    kw = dict(teacher_lse=cu["lse"], labels=cu["labels"], row_weights=cu["w"], workspace=ws)
    loss, grad = torch.empty(3, device="cuda"), torch.empty(3, 400, device="cuda")
    d.loss_grad(cu["x"], cu["ids"], cu["vals"], loss, grad, **kw)
    n = grad.norm(dim=1, keepdim=True)
    e = 2e-2

    def at(x):
        o = torch.empty(3, device="cuda")
        d.forward(x, cu["ids"], cu["vals"], o, **kw)
        return o.double()
    num = (at(cu["x"] + e * grad / n) - at(cu["x"] - e * grad / n)) / (2 * e)
    assert torch.allclose(num, n[:, 0].double(), rtol=1e-2)


@pytest.mark.parametrize("V,dt", [(20011, "f16"), (16390, "bf16"), (70001, "bf16"), (34003, "f32")])
def test_a_row_a_workgroup(lm, V, dt):
    """Rows enough for a workgroup each, of lengths either side of where its
    width changes (32 and 128 KB); a few of them padding."""
    c = make(131, V, 6, dt, 1.5, True, 0.3)
    c["w"][5:9] = 0
    run(lm, c, 1.5, 0.7, 0.3, "rows")


def test_a_row_a_workgroup_without_a_tail(lm):
    c = make(130, 17001, 40, "f32", 1.0, False, 0.0)
    c["ids"][3] = -1
    run(lm, c, 1.0, 1.0, 0.0, "rows without a tail")


def test_stats_of_padding_rows(lm):
    """Forward writes them all, in parts and as rows."""
    for rows in (4, 130):
        c = make(rows, 20000, 4, "bf16", 1.0, False, 0.0)
        c["w"][1] = 0
        d = lm.TopkDistill(20000, 4)
        loss, st = torch.full((rows,), 7.0, device="cuda"), torch.full((rows, 4), torch.nan, device="cuda")
        d.forward(c["x"].cuda(), c["ids"].cuda(), c["vals"].cuda(), loss, stats=st,
                  row_weights=c["w"].cuda(), workspace=d.workspace(rows))
        assert bool(st.isfinite().all()) and float(loss[1]) == 0 and not bool(st[1].any())
