"""Comparison of token-model outputs that holds infinities to their places.

lm_reference.check() takes an infinite expected value's tolerance, which is
infinite, for one: any number passes there.  Here an infinity has to be met by
the same infinity, and a number by a number, but where rounding alone decides:
a value within its tolerance of the largest that the type holds may round
either way.
"""
import torch


def check(got, want, what=""):
    """got: {name: tensor}; want: {name: (value, tolerance)}."""
    for name, g in got.items():
        v, tol = want[name]
        most = torch.finfo(g.dtype).max
        g = g.detach().cpu().double()
        assert g.shape == v.shape, f"{what} {name}: {tuple(g.shape)} for {tuple(v.shape)}"
        assert torch.equal(g.isnan(), v.isnan()), f"{what} {name}: NaNs differ"
        finite = v.isfinite()
        near = finite & (v.abs() + torch.where(finite, tol, 0) >= most) & (g == v.sign() * torch.inf)
        off = finite & ~near & ~((g - v).abs() <= tol)
        wrong = ~finite & ~v.isnan() & (g != v)
        bad = off | wrong
        if bool(bad.any()):
            at = tuple(int(i) for i in bad.nonzero()[0])
            raise AssertionError(f"{what} {name}: {int(bad.sum())} of {bad.numel()} off, first at "
                                 f"{at}: {float(g[at])!r} for {float(v[at])!r}, tolerance "
                                 f"{float(tol[at]):.3g}")
