"""GPU: a row that is not finite spoils its own gate's gradient and no other's,
however the rows of a gate are dealt to teams (block norms' backward)."""
import pytest
import torch

import lm_reference as ref
import lm_strict as strict
import test_lm_norm_gpu as base

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dh", "d_gate", "d_post_weight", "d_pre_weight")


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def backward(lm, c, D, post, pre, rpg, stats):
    norm = base.plan_of(lm, c, D, post, pre, 0.5)
    rows = len(c["x"])
    x, h, gate = (c[k].cuda() for k in ("x", "h", "gate"))
    o = dict(dx=torch.empty_like(x), dh=torch.empty_like(h), d_gate=torch.empty_like(gate),
             d_post_weight=torch.empty(D, device="cuda"), d_pre_weight=torch.empty(D, device="cuda"))
    norm.backward(c["dxo"].cuda(), c["dy"].cuda(), x, h, stats.cuda(), o["dx"], o["dh"], gate=gate,
                  rows_per_gate=rpg, workspace=norm.workspace(rows),
                  **{k: v for k, v in o.items() if k.startswith("d_")})
    return o


# gates of rows that their teams do not divide evenly (a team's last turns
# lie in the next gate's rows), for teams of a wave's part, of waves, and of a
# workgroup; gates of one row and of a few; teams without a row
@pytest.mark.parametrize("rows,D,rpg", [(1100, 1100, 100), (2600, 4096, 1301), (600, 5000, 299),
                                        (40000, 24, 4999), (3001, 1001, 1), (700, 300, 7)])
@pytest.mark.parametrize("kinds", [("layer", "layer"), ("rms", "rms")])
@pytest.mark.parametrize("what", ["nan", "constant"])
def test_a_bad_row_stays_with_its_gate(lm, rows, D, rpg, kinds, what):
    post, pre = kinds
    c = base.make(rows, D, "bf16", "bf16", post, pre, False, rpg)
    print(rows, D, rpg, kinds, what, flush=True)
    bad = [rpg, rows - 1]
    for r in bad:
        if what == "nan":
            c["x"][r] = torch.nan
            c["h"][r] = torch.nan
        else:       # without an eps, 1 / deviation is infinite
            c["x"][r] = c["h"][r] = 0.0
    stats = ref.stats_of(c["h"], c["x"], post, pre, base.EPS if what == "nan" else 0.0)
    o = backward(lm, c, D, post, pre, rpg, stats)
    want = ref.norm_backward(c["dxo"], c["dy"], c["x"], c["h"], stats, c["gate"], rpg, post, pre,
                             base.d64(c["pw"]), None, base.d64(c["qw"]), 0.5)
    strict.check({k: o[k] for k in NAMES}, want, f"rows={rows} D={D} rpg={rpg} {kinds} {what}")
    good = torch.ones(len(c["gate"]), dtype=torch.bool)
    good[[r // rpg for r in bad]] = False
    assert bool(o["d_gate"].cpu()[good].isfinite().all())
