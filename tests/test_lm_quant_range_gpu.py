"""GPU: the quantising norm on rows whose products with the weight are far from
one: their scales are ordinary numbers, since the norm's factor brings them back,
and every code has to be the nearest."""
import pytest
import torch

from lm_strict import check
from test_lm_quant_gpu import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def rows_of(size, D, res):
    """Rows whose largest are `size` (fp32), zeros among their elements."""
    h, x, w = make(9, D, "f32", "f32" if res else None)
    for t in (h, x) if res else (h,):
        t[:, 1::5] = 0
        t *= size / t.abs().amax(1, keepdim=True)
    return h, x, w


# (under eps 1e-6 the scale of a row of 5e-39 is 2^-126 or more for int8, not for e4m3)
@pytest.mark.parametrize("form", ["int8", "fp8"])
@pytest.mark.parametrize("size", [5e-39, 1e-37, 1e-36, 3e-34, 1e-28, 1e-20])
@pytest.mark.parametrize("D,group", [(5, 0), (300, 0), (300, 64), (512, 128), (600, 0), (4096, 0),
                                     (4096, 128), (8192, 0)])
def test_small_rows(lm, D, group, size, form):
    for res in (False, True):
        h, x, w = rows_of(size, D, res)
        q, s, _ = run(lm, h, x, w, form, group, f"size={size}")
        if size >= 1e-37 or form == "int8" and not res:
            assert bool((s.amax(1) > 0).all()) and bool(q.float().any(1).all())


@pytest.mark.parametrize("form", ["int8", "fp8"])
@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e25, 1e32])
@pytest.mark.parametrize("D,group", [(5, 0), (512, 128), (600, 0), (8192, 0)])
def test_small_and_large_weights(lm, D, group, size, form):
    """Ordinary rows under weights of such sizes."""
    h, x, w = make(9, D, "f32", "f32")
    run(lm, h, x, w * size, form, group, f"weight={size}")
    # and next to groups of ordinary ones
    w[: D // 2] *= size
    run(lm, h, x, w, form, group, f"weight={size} in part")


def test_a_row_small_and_a_row_large_at_once(lm):
    """Rows of one wave and of one workgroup that take different ways."""
    for D in (40, 300, 600, 1000):
        h, x, w = make(64, D, "f32", "f32")
        for t in (h, x):
            t[::3] *= 1e-37
            t[1::5] = 0
        for form in ("int8", "fp8"):
            for group in (0, 32):
                q, s, _ = run(lm, h, x, w, form, group)
                assert not bool(q[1::5].float().any()) and not bool(s[1::5].any())


@pytest.mark.parametrize("D", [5, 300, 600])
def test_where_squares_and_products_leave_fp32(lm, D):
    """What the definition says of them: no codes, and a scale that tells."""
    h, _, w = make(4, D, "f32", None)
    h[1] *= 1e25                       # squares past the range: as of an infinite row
    norm = lm.QuantNorm(D, weight=w.cuda(), form="int8")
    q, s = torch.ones(4, D, dtype=torch.int8, device="cuda"), torch.ones(4, 1, device="cuda")
    norm.forward(h.cuda(), q, s)
    assert float(s[1]) == 0 and not bool(q[1].any()) and bool(q[0].any())
    h[1] *= 1e-25
    w[2] = 3e38                        # a product past the range
    h[:, 2] = 5.0
    norm.weight = w.cuda()
    norm.forward(h.cuda(), q, s)
    assert bool((s == torch.inf).all()) and not bool(q.any())
    check({"q": q.float()}, {"q": (torch.zeros(4, D).double(), torch.zeros(4, D).double())})


@pytest.mark.parametrize("form", ["int8", "fp8"])
@pytest.mark.parametrize("size", [1e-20, 2e-19, 1e-12, 1e-6])
@pytest.mark.parametrize("D,group", [(300, 0), (4096, 0), (4096, 128)])
def test_small_rows_under_the_largest_weights(lm, D, group, size, form):
    """Products of ordinary size from both ends of the range, and large ones."""
    h, _, w = rows_of(size, D, False)
    w = w / w.abs().max() * 3e38
    run(lm, h, None, w, form, group, f"size={size}")
