"""GPU: block norms (forward, backward) against their fp64 definition, element
by element, over widths either side of every team shape, odd widths, gates
shared in every way rows can be dealt, mixed types, strides, in-place calls."""
import itertools

import pytest
import torch

import lm_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def make(rows, D, res, dt, post, pre, bias, rpg, seed=0, pdt=torch.float32):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(x=(3 * n(rows, D) + 0.2).to(DT[res]), h=(0.8 * n(rows, D) + 0.1).to(DT[dt]),
             gate=(0.5 * n((rows + rpg - 1) // rpg, D) + 0.5).to(DT[dt]) if rpg else None,
             dxo=n(rows, D).to(DT[res]), dy=n(rows, D).to(DT[dt]) if pre != "none" else None)
    for k, kind in (("p", post), ("q", pre)):
        c[k + "w"] = (1 + 0.2 * n(D)).to(pdt) if kind != "none" else None
        c[k + "b"] = (0.2 * n(D)).to(pdt) if bias and kind != "none" else None
    return c


def dev(t):
    return None if t is None else t.cuda()


def d64(t):
    return None if t is None else t.double()


def plan_of(lm, c, D, post, pre, scale):
    return lm.BlockNorm(D, post=post, pre=pre, post_weight=dev(c["pw"]), post_bias=dev(c["pb"]),
                        pre_weight=dev(c["qw"]), pre_bias=dev(c["qb"]), post_eps=EPS, pre_eps=EPS,
                        res_scale=scale)


def run_both(lm, rows, D, res="bf16", dt="bf16", post="rms", pre="rms", bias=False, rpg=0,
             scale=0.5, pdt=torch.float32, seed=0):
    c = make(rows, D, res, dt, post, pre, bias, rpg, seed, pdt)
    what = f"rows={rows} D={D} {res}/{dt} {post}/{pre} bias={bias} rpg={rpg}"
    print(what, flush=True)
    norm = plan_of(lm, c, D, post, pre, scale)
    x, h, gate = dev(c["x"]), dev(c["h"]), dev(c["gate"])
    xo = torch.full_like(x, 7.0)
    y = torch.full_like(h, 7.0) if pre != "none" else None
    st = torch.full((rows, 4), 7.0, device="cuda")
    norm.forward(x, h, xo, y, gate=gate, rows_per_gate=rpg, stats=st)
    want = ref.norm_forward(c["x"], c["h"], c["gate"], rpg, post, pre, d64(c["pw"]), d64(c["pb"]),
                            d64(c["qw"]), d64(c["qb"]), EPS, scale)
    got = dict(x_out=xo) if y is None else dict(x_out=xo, y=y)
    ref.check(got, want, "forward " + what)
    # the stats are those of h and of the unrounded x_out
    ws = ref.stats_of(c["h"], want["x_out"][0], post, pre, EPS)
    torch.testing.assert_close(st.cpu(), ws, rtol=1e-4, atol=1e-5)

    stats = ref.stats_of(c["h"], c["x"], post, pre, EPS)
    o = dict(dx=torch.full_like(x, 7.0), dh=torch.full_like(h, 7.0),
             d_gate=None if gate is None else torch.full_like(gate, 7.0))
    for k, on in (("d_post_weight", post != "none"), ("d_post_bias", bias and post != "none"),
                  ("d_pre_weight", pre != "none"), ("d_pre_bias", bias and pre != "none")):
        o[k] = torch.full((D,), 7.0, device="cuda") if on else None
    kw = {k: v for k, v in o.items() if k.startswith("d_")}
    norm.backward(dev(c["dxo"]), dev(c["dy"]), x, h, stats.cuda(), o["dx"], o["dh"], gate=gate,
                  rows_per_gate=rpg, workspace=norm.workspace(rows), **kw)
    want = ref.norm_backward(c["dxo"], c["dy"], c["x"], c["h"], stats, c["gate"], rpg, post, pre,
                             d64(c["pw"]), d64(c["pb"]), d64(c["qw"]), scale)
    ref.check({k: v for k, v in o.items() if v is not None}, want, "backward " + what)


# either side of each team width, odd widths, one column
@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 200, 256, 257, 500, 512, 513,
                               1001, 1024, 1025, 2048, 2050, 4095, 4096, 4097, 6000, 8191, 8192])
def test_widths(lm, D):
    run_both(lm, 5, D, post="layer", pre="rms", bias=True, rpg=2)
    run_both(lm, 3, D, res="f32", dt="f16", post="rms", pre="layer", rpg=0)


@pytest.mark.parametrize("post,pre", list(itertools.product(("none", "rms", "layer"), repeat=2)))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("D", [72, 1000])
def test_kinds(lm, post, pre, bias, D):
    run_both(lm, 9, D, post=post, pre=pre, bias=bias, rpg=3)
    run_both(lm, 9, D, post=post, pre=pre, bias=bias, rpg=0)


@pytest.mark.parametrize("res,dt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                    ("f16", "f16"), ("f32", "f16")])
@pytest.mark.parametrize("D", [33, 768, 5000])
@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16, torch.float16])
def test_types(lm, res, dt, D, pdt):
    run_both(lm, 6, D, res=res, dt=dt, post="rms", pre="layer", bias=True, rpg=6, pdt=pdt)
    run_both(lm, 6, D, res=res, dt=dt, post="layer", pre="rms", bias=True, rpg=1, pdt=pdt)


# how rows share gates: one each, few, a gate to several teams, one for all,
# more rows a gate than there are rows; the last gate cut short
@pytest.mark.parametrize("rpg", [0, 1, 2, 3, 7, 64, 100, 333, 1999, 2000, 10**9])
@pytest.mark.parametrize("rows,D", [(2000, 24), (1500, 160), (1100, 1100)])
def test_gates(lm, rows, D, rpg):
    run_both(lm, rows, D, post="layer", pre="rms", bias=True, rpg=rpg)


@pytest.mark.parametrize("rpg", [1, 700, 1300, 2600])
def test_gates_over_many_teams(lm, rpg):
    # more than two rows a team: 1024 workgroup-wide teams
    run_both(lm, 2600, 4096, res="bf16", post="rms", pre="rms", rpg=rpg)


@pytest.mark.parametrize("rows", [1, 2, 255, 257, 1030])
def test_row_counts(lm, rows):
    run_both(lm, rows, 300, rpg=rows)


def test_no_rows(lm):
    D = 40
    c = make(0, D, "f32", "bf16", "rms", "layer", True, 1)
    norm = plan_of(lm, c, D, "rms", "layer", 1.0)
    x, h = dev(c["x"]), dev(c["h"])
    norm.forward(x, h, x.clone(), h.clone())
    o = {k: torch.full((D,), 7.0, device="cuda")
         for k in ("d_post_weight", "d_post_bias", "d_pre_weight", "d_pre_bias")}
    norm.backward(x, h, x, h, torch.zeros(0, 4, device="cuda"), x.clone(), h.clone(),
                  workspace=norm.workspace(0), **o)
    for v in o.values():
        assert float(v.abs().max()) == 0


def test_strides_in_place_and_wanted_sums(lm):
    rows, D, W = 37, 250, 611
    c = make(rows, D, "bf16", "bf16", "rms", "rms", False, 5)
    norm = plan_of(lm, c, D, "rms", "rms", 1.0)

    def wide(t, at):   # the columns [at, at + D) of wider rows
        w = torch.full((t.shape[0], W), 3.0, dtype=t.dtype, device="cuda")
        w[:, at:at + D] = t.cuda()
        return w, w[:, at:at + D]

    x, h, gate = dev(c["x"]), dev(c["h"]), dev(c["gate"])
    xo, y = torch.empty_like(x), torch.empty_like(h)
    norm.forward(x, h, xo, y, gate=gate, rows_per_gate=5)
    wx, vx = wide(c["x"], 1)
    wh, vh = wide(c["h"], 301)
    wg, vg = wide(c["gate"], 17)
    norm.forward(vx, vh, vx, vh, gate=vg, rows_per_gate=5)   # in place, odd strides
    assert torch.equal(vx, xo) and torch.equal(vh, y)
    for w, at in ((wx, 1), (wh, 301)):                        # nothing beside the columns
        assert bool((w[:, :at] == 3).all()) and bool((w[:, at + D:] == 3).all())

    stats = ref.stats_of(c["h"], c["x"], "rms", "rms", EPS).cuda()
    ws = norm.workspace(rows)
    dx, dh, dg = torch.empty_like(x), torch.empty_like(h), torch.empty_like(gate)
    w1, w2 = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    args = (dev(c["dxo"]), dev(c["dy"]), x, h, stats)
    norm.backward(*args, dx, dh, gate=gate, rows_per_gate=5, d_gate=dg, d_post_weight=w1,
                  d_pre_weight=w2, workspace=ws)
    wdx, vdx = wide(c["dxo"], 3)
    wdy, vdy = wide(c["dy"], 9)
    only = torch.empty(D, device="cuda")
    norm.backward(vdx, vdy, x, h, stats, vdx, vdy, gate=gate, rows_per_gate=5,
                  d_pre_weight=only, workspace=ws)            # dx over dx_out, dh over dy
    assert torch.equal(vdx, dx) and torch.equal(vdy, dh) and torch.equal(only, w2)
    assert bool((wdx[:, :3] == 3).all()) and bool((wdy[:, 9 + D:] == 3).all())


def test_differences(lm):
    """The backward's dx, dh and d_gate against differences of the forward (fp32):
    along a direction, (f(v + e d) - f(v - e d)) / 2e is off by e^2 times third
    derivatives (below 1e-2 of the value at e = 1e-2) and by 1e-4 or so of the
    fp32 sums' rounding over e."""
    rows, D, rpg = 6, 90, 4
    c = make(rows, D, "f32", "f32", "layer", "rms", True, rpg)
    norm = plan_of(lm, c, D, "layer", "rms", 0.5)
    x, h, gate = dev(c["x"]), dev(c["h"]), dev(c["gate"])
    dxo, dy = dev(c["dxo"]), dev(c["dy"])
    xo, y, st = torch.empty_like(x), torch.empty_like(h), torch.empty(rows, 4, device="cuda")
    norm.forward(x, h, xo, y, gate=gate, rows_per_gate=rpg, stats=st)
    o = dict(x=torch.empty_like(x), h=torch.empty_like(h), gate=torch.empty_like(gate))
    norm.backward(dxo, dy, xo, h, st, o["x"], o["h"], gate=gate, rows_per_gate=rpg,
                  d_gate=o["gate"], workspace=norm.workspace(rows))
    at = dict(x=x, h=h, gate=gate)

    def value(v):
        a, b = torch.empty_like(x), torch.empty_like(h)
        norm.forward(v["x"], v["h"], a, b, gate=v["gate"], rows_per_gate=rpg)
        return float((a.double() * dxo.double()).sum() + (b.double() * dy.double()).sum())

    for k in at:
        d = o[k] / o[k].norm()     # along the gradient, the slope is its length
        e = 1e-2
        num = (value({**at, k: at[k] + e * d}) - value({**at, k: at[k] - e * d})) / (2 * e)
        assert abs(num - float(o[k].norm())) < 1e-2 * float(o[k].norm()), k


def test_same_bits_again(lm):
    rows, D = 900, 1000
    c = make(rows, D, "bf16", "bf16", "rms", "rms", False, rows)
    norm = plan_of(lm, c, D, "rms", "rms", 1.0)
    stats = ref.stats_of(c["h"], c["x"], "rms", "rms", EPS).cuda()
    x, h, gate = dev(c["x"]), dev(c["h"]), dev(c["gate"])
    outs = []
    for _ in range(2):
        o = [torch.empty_like(x), torch.empty_like(h), torch.empty_like(gate),
             torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]
        norm.backward(dev(c["dxo"]), dev(c["dy"]), x, h, stats, o[0], o[1], gate=gate,
                      rows_per_gate=rows, d_gate=o[2], d_post_weight=o[3], d_pre_weight=o[4],
                      workspace=norm.workspace(rows))
        outs.append(o)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
