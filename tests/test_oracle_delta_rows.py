"""The gated delta rule's oracle at rows of zeros, and nearly so, that the call
normalises."""
import numpy as np
import pytest

from oracle import delta


def _case(seed, size):
    r = np.random.default_rng(seed)
    b, l, h, g, n, p = 2, 6, 4, 2, 5, 3
    c = dict(q=r.normal(size=(b, l, g, n)), k=r.normal(size=(b, l, g, n)),
             v=r.normal(size=(b, l, h, p)), dt=r.normal(size=(b, l, h)),
             A=-np.exp(r.normal(size=h)), beta=r.uniform(0, 1, size=(b, l, h)),
             dt_bias=r.normal(size=h) * 0.3)
    c["q"][:, ::2] *= size
    c["k"][:, 1::3] *= size
    return c, r.normal(size=c["v"].shape)


@pytest.mark.parametrize("size", [0.0, 1e-25, 1e-3])
def test_gradient_of_small_rows_against_differences(size):
    """Central differences of a step of 1e-4 sqrt(eps): off by 1e-8 of the third
    derivatives (a row's are of the first's size in units of sqrt(eps)), roundings
    by less; 1e-6 of the largest entry allows both."""
    c, dy = _case(3, size)
    kw = dict(normalize=True, norm_eps=1e-2)
    got = delta.grad(**c, dy=dy, **kw)
    for out, name in (("dq", "q"), ("dk", "k")):
        want = np.empty(c[name].shape)
        for at in np.ndindex(want.shape):
            ends = []
            for e in (1e-5, -1e-5):
                x = c[name].copy()
                x[at] += e
                ends.append((delta.scan(**{**c, name: x}, **kw)["y"] * dy).sum())
            want[at] = (ends[0] - ends[1]) / 2e-5
        np.testing.assert_allclose(got[out], want, atol=1e-6 * np.abs(want).max(), err_msg=out)
        rows = want[:, ::2] if name == "q" else want[:, 1::3]
        assert np.abs(rows).max() > 0.1


def test_rows_of_zeros_without_eps():
    """No derivative there: the rows stay zeros and take none."""
    c, dy = _case(4, 0.0)
    got = delta.grad(**c, dy=dy, normalize=True, norm_eps=0.0)
    assert (got["dq"][:, ::2] == 0).all() and (got["dk"][:, 1::3] == 0).all()
    assert np.isfinite(got["dq"]).all() and np.isfinite(got["dk"]).all()
