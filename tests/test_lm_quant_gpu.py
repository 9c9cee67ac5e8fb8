"""GPU: the quantising norm against its fp64 definition: sums, scales, and every
code the nearest."""
import pytest
import torch

import lm_step_reference as ref
from lm_reference import U, half_step
from lm_strict import check

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def make(rows, D, dt, rt, wt="f32", seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    h = n(rows, D)
    h[:, ::37] *= 10
    return h.to(DT[dt]), None if rt is None else (3 * n(rows, D)).to(DT[rt]), \
        (1 + 0.2 * n(D)).to(DT[wt])


def run(lm, h, x, w, form, group, what=""):
    rows, D = h.shape
    what += f" rows={rows} D={D} {h.dtype} {None if x is None else x.dtype} {form} {group}"
    print(what, flush=True)
    norm = lm.QuantNorm(D, weight=w.cuda(), form=form, group=group, eps=EPS)
    q = torch.full((rows, D), 3.0, device="cuda").to(lm.CODE[form][1])
    scales = torch.full((rows, norm.groups), 9.0, device="cuda")
    stats = torch.full((rows, 4), 9.0, device="cuda")
    rt = h.dtype if x is None else x.dtype
    x_out = torch.full((rows, D), 9.0, dtype=rt, device="cuda")
    norm.forward(h.cuda(), q, scales, x=None if x is None else x.cuda(), x_out=x_out, stats=stats)
    t, mag, v, tv, s, ts = ref.quant_norm(h, x, w, EPS, form, group)
    check({"x_out": x_out, "scales": scales},
          {"x_out": (t, half_step(t, rt) + U * mag), "scales": (s, ts)}, what)
    ref.check_codes(q.cpu(), scales.cpu(), v, tv, form, group, what)
    st = stats.cpu().double()
    assert bool((st[:, :3] == torch.tensor([0.0, 1.0, 0.0])).all())
    rs = 1 / ((t * t).mean(1) + EPS).sqrt()
    assert bool(((st[:, 3] - rs).abs() <= 40 * U * rs * (1 + rs * (mag * mag).mean(1).sqrt())).all())
    return q, scales, x_out


@pytest.mark.parametrize("form", ["int8", "fp8"])
@pytest.mark.parametrize("dt,rt", [("f32", None), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                   ("f16", None), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 65, 300, 512, 520, 1001, 4096, 8192])
def test_widths_and_types(lm, D, dt, rt, form):
    h, x, w = make(9, D, dt, rt, wt=dt)
    run(lm, h, x, w, form, 0)
    run(lm, h, x, w, form, 64)


@pytest.mark.parametrize("group", [32, 64, 128, 256, 512])
@pytest.mark.parametrize("D", [5, 31, 32, 40, 128, 500, 511, 513, 1500, 4100])
def test_groups(lm, D, group):
    h, x, w = make(6, D, "bf16", "bf16")
    run(lm, h, x, w, "fp8", group)
    run(lm, h, x, w, "int8", group)


@pytest.mark.parametrize("rows", [1, 2, 31, 33, 1500, 9000])
def test_rows(lm, rows):
    for D in (40, 600):
        h, x, w = make(rows, D, "bf16", "f32")
        run(lm, h, x, w, "fp8", 128)
        run(lm, h, x, w, "int8", 0)


def test_nothing_and_tiny(lm):
    """Rows of zeros; groups of zeros; scales below the smallest normal."""
    h, _, w = make(4, 256, "f32", None)
    h[0] = 0
    h[1, 128:] = 0
    h[2, :128] *= 1e-37
    for form in ("int8", "fp8"):
        q, s, _ = run(lm, h, None, w, form, 128)
        assert not bool(s[0].any()) and float(s[1, 1]) == 0
        # the largest of the tiny ones, 1.82e-36: over 127 above 2^-126, over 448 below it
        assert (float(s[2, 0]) == 0) == (form == "fp8")
        assert not bool(q[0].float().any())


@pytest.mark.parametrize("form", ["int8", "fp8"])
def test_not_finite(lm, form):
    h, x, w = make(8, 512, "f32", "f32")
    h[1, 200] = torch.nan
    x[2, 300] = torch.inf
    h[3, 5], x[3, 5] = torch.inf, -torch.inf
    norm = lm.QuantNorm(512, weight=w.cuda(), form=form, group=128)
    clean = lambda: (torch.empty(8, 512, device="cuda").to(lm.CODE[form][1]),  # noqa: E731
                     torch.empty(8, 4, device="cuda"))
    q, s = clean()
    norm.forward(h.cuda(), q, s, x=x.cuda())
    s, q = s.cpu(), q.float().cpu()
    assert bool(s[1].isnan().all()) and bool((q[1] == 0).all())     # the row's norm is no number
    assert bool(s[3].isnan().all())
    assert bool(s[2, 2].isnan()) and bool((s[2, [0, 1, 3]] == 0).all()) and bool((q[2] == 0).all())
    h[1, 200] = 0
    x[2, 300] = 0
    h[3, 5] = x[3, 5] = 0
    q2, s2 = clean()
    norm.forward(h.cuda(), q2, s2, x=x.cuda())
    rest = [0, 4, 5, 6, 7]
    assert torch.equal(q[rest], q2.float().cpu()[rest]) and torch.equal(s[rest], s2.cpu()[rest])


def test_strides_and_places(lm):
    rows, D = 21, 203
    h, x, w = make(rows, D, "bf16", "bf16")
    q, s, xo = run(lm, h, x, w, "int8", 32)
    norm = lm.QuantNorm(D, weight=w.cuda(), form="int8", group=32, eps=EPS)

    def wide(t, at, W):
        b = torch.full((rows, W), 3, dtype=t.dtype, device="cuda")
        b[:, at:at + t.shape[1]] = t.cuda()
        return b, b[:, at:at + t.shape[1]]
    for at, W in ((0, 256), (1, 211), (3, 300)):
        (wq, q2), (wx, xo2), (wsc, s2) = wide(torch.zeros_like(q), at, W), \
            wide(torch.zeros_like(xo), at, W), wide(torch.zeros_like(s), at, W)
        norm.forward(wide(h, at, W)[1], q2, s2, x=wide(x, at, W)[1], x_out=xo2)
        assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(xo2, xo)
        for b, n in ((wq, D), (wx, D), (wsc, s.shape[1])):
            assert bool((b[:, :at] == 3).all()) and bool((b[:, at + n:] == 3).all())
    for place in ("x", "h"):
        hc, xc, q2, s2 = h.cuda(), x.cuda(), torch.empty_like(q), torch.empty_like(s)
        norm.forward(hc, q2, s2, x=xc, x_out=xc if place == "x" else hc)
        assert torch.equal(xc if place == "x" else hc, xo) and torch.equal(q2, q) and torch.equal(s2, s)


def test_fp8_ties_and_range(lm):
    """Values that fall between two codes go to the even one, as torch rounds."""
    c = torch.arange(0, 449).float() / 1.0
    h = torch.cat([c, c + 0.5, c / 64, -c / 256])[None]
    h = h[:, :1792]
    w = torch.ones(h.shape[1])
    norm = lm.QuantNorm(h.shape[1], weight=w.cuda(), form="fp8")
    q, s = torch.empty(h.shape, device="cuda").to(torch.float8_e4m3fn), torch.empty(1, 1, device="cuda")
    st = torch.empty(1, 4, device="cuda")
    norm.forward(h.cuda(), q, s, stats=st)
    v = h.cuda() * st[0, 3]
    assert torch.equal(q.float(), (v / s).clamp(-448, 448).to(torch.float8_e4m3fn).float())


def test_straight_through_gradient(lm):
    """Its stats are what a block norm without a post norm reads."""
    rows, D = 12, 320
    h, x, w = make(rows, D, "f32", "f32")
    norm = lm.QuantNorm(D, weight=w.cuda(), form="fp8", eps=EPS)
    q, s = torch.empty(rows, D, device="cuda").to(torch.float8_e4m3fn), torch.empty(rows, 1, device="cuda")
    st, xo = torch.empty(rows, 4, device="cuda"), torch.empty(rows, D, device="cuda")
    norm.forward(h.cuda(), q, s, x=x.cuda(), x_out=xo, stats=st)
    block = lm.BlockNorm(D, post="none", pre="rms", pre_weight=w.cuda(), pre_eps=EPS)
    y, st2, xo2 = torch.empty_like(xo), torch.empty_like(st), torch.empty_like(xo)
    block.forward(x.cuda(), h.cuda(), xo2, y, stats=st2)
    assert torch.equal(xo, xo2)
    # a step of the codes' (2^-4 of a value, 2^-10 of the scale) and both norms' errors
    assert bool(((q.float() * s - y).abs() <= y.abs() * (2.0 ** -4 + 1e-5) + s * 2.0 ** -10).all())
    grads = []
    for stats in (st, st2):
        dx, dh, dw = torch.empty_like(xo), torch.empty_like(xo), torch.empty(D, device="cuda")
        block.backward(torch.zeros_like(xo), y, xo, h.cuda(), stats, dx, dh, d_pre_weight=dw,
                       workspace=block.workspace(rows))
        grads.append((dx, dh, dw))
    for a, b in zip(*grads):
        # the stats differ by roundings of the same sum: 40 U of what they scale
        assert bool(((a - b).abs() <= 200 * U * (b.abs() + b.abs().max())).all())


def test_no_rows(lm):
    norm = lm.QuantNorm(16, weight=torch.ones(16, device="cuda"))
    norm.forward(torch.empty(0, 16, device="cuda"), torch.empty(0, 16, dtype=torch.int8, device="cuda"),
                 torch.empty(0, 1, device="cuda"))
