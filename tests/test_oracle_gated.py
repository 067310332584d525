"""The oracles of the linear layer and of the gated recurrence: closed forms,
and gradients against central differences."""
import numpy as np
import pytest

from oracle import gated, linear


def _case(seed, b, l, d, docs=True):
    rng = np.random.default_rng(seed)
    lam = rng.normal(size=d) - 3
    seq = np.cumsum(rng.random((b, l)) < 0.2, 1).astype(np.int32) if docs else None
    return dict(x=rng.normal(size=(b, l, d)), gates=2 * rng.normal(size=(b, l, 2 * d)), lam=lam,
                init=rng.normal(size=(b, d))), seq, rng


def test_scan_is_its_closed_form():
    """h_t = sum_j (prod_{j<k<=t} a_k) v_j + (prod a) h_0."""
    c, _, _ = _case(1, 2, 9, 3, docs=False)
    r = gated.scan(c["x"], c["gates"], c["lam"], 8.0, c["init"])
    d = 3
    u = 8.0 * np.log1p(np.exp(c["lam"])) / (1 + np.exp(-c["gates"][..., :d]))
    v = np.sqrt(1 - np.exp(-2 * u)) / (1 + np.exp(-c["gates"][..., d:])) * c["x"]
    for t in range(9):
        want = np.exp(-u[:, :t + 1].sum(1)) * c["init"]
        for j in range(t + 1):
            want = want + np.exp(-u[:, j + 1:t + 1].sum(1)) * v[:, j]
        np.testing.assert_allclose(r["y"][:, t], want, rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(r["final"], r["y"][:, -1])


def test_documents_equal_separate_sequences():
    c, _, _ = _case(2, 1, 20, 4, docs=False)
    seq = np.array([[5] * 7 + [1] + [5] * 12], np.int32)
    r = gated.scan(c["x"], c["gates"], c["lam"], 8.0, c["init"], seq)
    for lo, hi, h0 in ((0, 7, c["init"]), (7, 8, None), (8, 20, None)):
        s = gated.scan(c["x"][:, lo:hi], c["gates"][:, lo:hi], c["lam"], 8.0, h0)
        np.testing.assert_allclose(r["y"][:, lo:hi], s["y"], rtol=1e-13)


@pytest.mark.parametrize("docs", [False, True])
def test_scan_gradient_against_differences(docs):
    c, seq, rng = _case(3, 2, 6, 3, docs)
    dy, df = rng.normal(size=(2, 6, 3)), rng.normal(size=(2, 3))

    def loss(**over):
        k = dict(c, **over)
        r = gated.scan(k["x"], k["gates"], k["lam"], 8.0, k["init"], seq)
        return (r["y"] * dy).sum() + (r["final"] * df).sum()

    g = gated.grad(c["x"], c["gates"], c["lam"], 8.0, dy, c["init"], seq, df)
    for name, key in (("x", "dx"), ("gates", "dgates"), ("lam", "dlam"), ("init", "d_init")):
        it = np.nditer(c[name], flags=["multi_index"])
        for _ in it:
            p, m = c[name].copy(), c[name].copy()
            p[it.multi_index] += 1e-5
            m[it.multi_index] -= 1e-5
            num = (loss(**{name: p}) - loss(**{name: m})) / 2e-5
            np.testing.assert_allclose(g[key][it.multi_index], num, rtol=2e-6, atol=1e-8)


@pytest.mark.parametrize("name", ["none", "silu", "gelu", "sigmoid"])
def test_linear_gradient_against_differences(name):
    rng = np.random.default_rng(4)
    x, w, b = rng.normal(size=(3, 4)), rng.normal(size=(5, 4)), rng.normal(size=5)
    dy = rng.normal(size=(3, 5))
    _, pre = linear.linear(x, w, b, name)
    g = linear.linear_grad(dy, x, w, pre, name)
    for arr, key in ((x, "dx"), (w, "dweight"), (b, "dbias")):
        it = np.nditer(arr, flags=["multi_index"])
        for _ in it:
            v = arr[it.multi_index]
            out = []
            for s in (1e-5, -1e-5):
                arr[it.multi_index] = v + s
                out.append((linear.linear(x, w, b, name)[0] * dy).sum())
            arr[it.multi_index] = v
            np.testing.assert_allclose(g[key][it.multi_index], (out[0] - out[1]) / 2e-5, rtol=2e-6,
                                       atol=1e-8)
