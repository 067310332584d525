"""The fp64 oracle of the gated delta rule and of the layer norm: hand-worked
cases, invariants, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import delta


def _case(seed, b=2, l=9, h=4, g=2, n=5, p=3, packed=True, init=True):
    r = np.random.default_rng(seed)
    c = dict(q=r.normal(size=(b, l, g, n)), k=r.normal(size=(b, l, g, n)) / np.sqrt(n),
             v=r.normal(size=(b, l, h, p)), dt=r.normal(size=(b, l, h)),
             A=-np.exp(r.normal(size=h)), beta=r.uniform(0, 1, size=(b, l, h)),
             dt_bias=r.normal(size=h) * 0.3)
    c["init"] = r.normal(size=(b, h, n, p)) if init else None
    c["seq"] = np.cumsum(r.random((b, l)) < 0.3, 1).astype(np.int32) if packed else None
    return c, r


def test_one_token_from_zero():
    """S = beta k v^T, y = scale (q . k) beta v."""
    c, _ = _case(1, l=1, packed=False, init=False)
    r = delta.scan(**c, scale=0.7)
    k, q = np.repeat(c["k"], 2, 2)[:, 0], np.repeat(c["q"], 2, 2)[:, 0]
    bv = c["beta"][:, 0, :, None] * c["v"][:, 0]
    np.testing.assert_allclose(r["final"], k[..., None] * bv[:, :, None], atol=1e-14)
    np.testing.assert_allclose(r["y"][:, 0], 0.7 * (q * k).sum(-1)[..., None] * bv, atol=1e-14)


def test_full_strength_replaces_what_a_key_holds():
    """beta = 1 and a unit key without decay: reading with the key gives v."""
    c, _ = _case(2, packed=False)
    c["A"] = np.zeros(4)
    c["beta"] = np.ones_like(c["beta"])
    c["q"] = c["k"]
    r = delta.scan(**c, scale=1.0, normalize=True, norm_eps=0.0)
    np.testing.assert_allclose(r["y"], c["v"], atol=1e-12)


def test_documents_are_independent():
    c, _ = _case(3, b=1, l=12)
    c["seq"] = np.array([[0] * 5 + [1] * 7], np.int32)
    whole = delta.scan(**c)["y"]
    cut = lambda lo, hi: {k: (v[:, lo:hi] if k in ("q", "k", "v", "dt", "beta") else v)  # noqa: E731
                          for k, v in c.items() if k != "seq"}
    first, second = cut(0, 5), cut(5, 12)
    second["init"] = None
    np.testing.assert_array_equal(whole[:, :5], delta.scan(**first)["y"])
    np.testing.assert_allclose(whole[:, 5:], delta.scan(**second)["y"], atol=1e-14)


def test_steps_continue_a_scan():
    c, _ = _case(4, packed=False)
    whole = delta.scan(**c)
    st = c["init"]
    for t in range(9):
        y, st = delta.step(st, *(c[k][:, t] for k in ("q", "k", "v", "dt")), c["A"],
                           c["beta"][:, t], dt_bias=c["dt_bias"])
        np.testing.assert_allclose(y, whole["y"][:, t], atol=1e-13)
    np.testing.assert_allclose(st, whole["final"], atol=1e-13)


@pytest.mark.parametrize("normalize,packed,init", [(False, False, True), (True, True, True),
                                                   (True, False, False)])
def test_gradient_against_differences(normalize, packed, init):
    """Central differences of step 1e-5: off by about 1e-10 of third derivatives
    and 1e-11 of roundings; 1e-6 of the largest entry allows both."""
    c, r = _case(5, l=6, packed=packed, init=init)
    kw = dict(normalize=normalize, norm_eps=1e-3, dt_limit=(0.2, 1.5))
    dy, df = r.normal(size=c["v"].shape), r.normal(size=(2, 4, 5, 3))

    def loss(c):
        o = delta.scan(**c, **kw)
        return (o["y"] * dy).sum() + (o["final"] * df).sum()
    got = delta.grad(**c, dy=dy, d_final=df, **kw)
    names = dict(dq="q", dk="k", dv="v", ddt="dt", dbeta="beta", dA="A", ddt_bias="dt_bias")
    if init:
        names["d_init"] = "init"
    for out, name in names.items():
        want = np.empty(c[name].shape)
        for at in np.ndindex(want.shape):
            ends = []
            for e in (1e-5, -1e-5):
                x = c[name].copy()
                x[at] += e
                ends.append(loss({**c, name: x}))
            want[at] = (ends[0] - ends[1]) / 2e-5
        np.testing.assert_allclose(got[out], want, atol=1e-6 * max(1.0, np.abs(want).max()),
                                   err_msg=out)


def test_layer_norm_gradient_against_differences():
    r = np.random.default_rng(6)
    x, w, b, dy, ds = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=7), \
        r.normal(size=(3, 7)), r.normal(size=(3, 7))
    got = delta.layer_norm_grad(dy, x, w, eps=0.1, d_sum=ds)
    loss = lambda x, w, b: (delta.layer_norm(x, w, b, eps=0.1)[0] * dy).sum()  # noqa: E731
    for i, name in enumerate(("dx", "dweight", "dbias")):
        args = [x, w, b]
        want = np.empty(args[i].shape)
        for at in np.ndindex(want.shape):
            ends = []
            for e in (1e-5, -1e-5):
                a = [t.copy() for t in args]
                a[i][at] += e
                ends.append(loss(*a))
            want[at] = (ends[0] - ends[1]) / 2e-5
        np.testing.assert_allclose(got[name], want + (ds if name == "dx" else 0), atol=1e-8)


def test_layer_norm_of_constant_rows():
    y, mean, rstd = delta.layer_norm(np.full((2, 4), 3.0), None, np.arange(4.0), eps=1e-4)
    np.testing.assert_array_equal(y, np.tile(np.arange(4.0), (2, 1)))
    np.testing.assert_allclose(rstd, 100.0)
