"""The gated recurrence away from decays near one: strong decays (rates up to
90), rates near the bottom of fp32 and rates without bound, against the fp64
oracle in oracle/gated.py.

Tolerances, per element, in units of 2^-24.  Gates are cut at +-8, so a
sigmoid is off by 14 (its exponential's argument 8 x 1.5, the exponential, the
sum and the reciprocal), the rate u by 24 (softplus and two products 10 more)
and a decay e^-u by 24 u + 4.  1 - a^2 takes 24 from u (2u / (e^2u - 1) <= 1)
and at most 40 from the subtraction, which starts at 2u = 1/8; its square root
half of that, so an added value is off by at most 50.  a^2 u / beta is off by
48 u + 80.  delta = 2^-18 is 64 units: it covers a decay with max(1, u) delta, an
added value with delta, and the gradient's terms with 4 max(1, u) delta, which is
how the oracle takes it through the recurrence and the gradient to first
order.  An output in bf16 adds half a step, 2^-8 of its value.  1e-30 stands for
what underflows.
"""
import numpy as np
import pytest

from gpu_util import log, to_f64, torch_mod

pytestmark = pytest.mark.gpu

DELTA = 2.0 ** -18
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 1e-30


def _case(seed, b, l, d, io, lam, docs=False, init=True):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32

    def t(a):
        return torch.from_numpy(a.astype(np.float32)).to("cuda")
    seq = None
    if docs:
        seq = torch.from_numpy(np.cumsum(rng.random((b, l)) < 0.1, 1).astype(np.int32)).to("cuda")
    return dict(x=t(rng.normal(size=(b, l, d))).to(dt),
                gates=t(np.clip(3 * rng.normal(size=(b, l, 2 * d)), -8, 8)).to(dt),
                lam=t(np.linspace(*lam, d)), init=t(rng.normal(size=(b, d))) if init else None,
                seq=seq, dy=t(rng.normal(size=(b, l, d))).to(dt), dfin=t(rng.normal(size=(b, d))))


def _np(c):
    return {k: None if v is None else (v.cpu().numpy() if k == "seq" else to_f64(v))
            for k, v in c.items()}


def _close(g, o, tol, what):
    g = to_f64(g)
    assert g.shape == o.shape, (what, g.shape, o.shape)
    assert np.isfinite(g).all(), what
    err = np.abs(g - o) - tol
    assert (err <= 0).all(), "%s: %d of %d outside, worst excess %.3g at %s (got %r, want %r)" % (
        what, int((err > 0).sum()), err.size, err.max(), np.unravel_index(err.argmax(), err.shape),
        g.flat[err.argmax()], o.flat[err.argmax()])


def _compare(c, io, scale, with_final=True, tiny=TINY):
    """Forward, gradient (from kept states and without) and decode steps."""
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import gated as go
    torch = torch_mod()
    n, half = _np(c), HALF[io]
    kw = dict(scale=scale, initial_state=c["init"], seq_idx=c["seq"])
    y, fin, st = ssd.gated_scan(c["x"], c["gates"], c["lam"], return_final_state=True,
                                return_states=True, **kw)
    dfin = c["dfin"] if with_final else None
    grads = [ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], d_final=dfin, states=s, **kw)
             for s in (None, st)]
    torch.cuda.synchronize()
    r = go.scan(n["x"], n["gates"], n["lam"], scale, n["init"], n["seq"], delta=DELTA)
    _close(y, r["y"], r["err"] + half * 1.01 * np.abs(r["y"]) + tiny, "y")
    _close(fin, r["final"], r["err"][:, -1] + 2.0 ** -24 * np.abs(r["final"]) + tiny, "final")
    k = go.grad(n["x"], n["gates"], n["lam"], scale, n["dy"], n["init"], n["seq"],
                n["dfin"] if with_final else None, delta=DELTA)
    d = c["lam"].shape[0]
    for g in grads:
        _close(g["dx"], k["dx"], k["err_dx"] + half * 1.01 * np.abs(k["dx"]) + tiny, "dx")
        for what, s in (("dr", slice(0, d)), ("di", slice(d, None))):
            o = k["dgates"][..., s]
            _close(g["dgates"][..., s], o,
                   k["err_dgates"][..., s] + half * 1.01 * np.abs(o) + tiny, what)
        _close(g["dlam"], k["dlam"], k["err_dlam"] + tiny, "dlam")
        if "d_init" in g:
            _close(g["d_init"], k["d_init"],
                   k["err_d_init"] + 2.0 ** -23 * np.abs(k["d_init"]) + tiny, "d_init")
    if c["seq"] is None:
        state = torch.zeros_like(c["dfin"]) if c["init"] is None else c["init"].clone()
        for t in range(min(3, c["x"].shape[1])):
            ys = ssd.gated_step(state, c["x"][:, t].contiguous(), c["gates"][:, t].contiguous(),
                                c["lam"], scale=scale)
            torch.cuda.synchronize()
            o, e = r["y"][:, t], r["err"][:, t]
            _close(ys, o, e + half * 1.01 * np.abs(o) + tiny, "step")
            _close(state, o, e + 2.0 ** -24 * np.abs(o) + tiny, "step's state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("docs,init", [(False, True), (False, False), (True, True), (True, False)])
@pytest.mark.parametrize("shape,scale", [((2, 1, 64), 8.0), ((3, 70, 33), 8.0), ((1, 300, 128), 8.0),
                                         ((2, 200, 66), 1.5), ((2, 130, 40), 30.0)], ids=str)
def test_strong_decays(shape, scale, docs, init, io):
    """Rates from scale softplus(-8) to scale softplus(3)."""
    log("strong decays", shape, scale, docs, init, io)
    c = _case(6000 + shape[1], *shape, io=io, lam=(-8.0, 3.0), docs=docs, init=init)
    _compare(c, io, scale, with_final=shape[1] != 70)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("init", [False, True])
def test_rates_near_the_bottom(init, io):
    """Rates from 8 e^-82 to 8 e^-60: 1 - a^2 down to 1e-36, its square root, which
    the gradient divides by, down to 1e-18; nothing but fp32's smallest normal
    value is taken for zero.  Gates from -2, so that every product stays normal."""
    log("rates near the bottom", init, io)
    c = _case(6100, 2, 70, 46, io, lam=(-82.0, -60.0), init=init)
    c["gates"] = c["gates"].clamp(min=-2)
    _compare(c, io, 8.0, tiny=2.0 ** -126)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("l", [1, 40, 300])
@pytest.mark.parametrize("docs", [False, True])
def test_gradient_of_rates_without_bound(docs, l, io):
    """lam = inf, lam so far out that scale softplus(lam) overflows, and a rate that
    overflows only in binary orders: the decay is zero and stays zero, so the
    decay gate, lam and the initial state have zero gradients and x and the
    other gate those of y = sigmoid(i) x; a NaN stays in its channel.  With
    scale = 0 nothing decays, whatever lam."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    log("rates without bound", docs, l, io)
    for scale, ends in ((8.0, [np.inf, 1e38, 3e37]), (1e30, [np.inf, 1e9, 5.0])):
        c = _case(6200 + l, 2, l, 6, io, lam=(-3.0, -2.0), docs=docs)
        lam = c["lam"]
        lam[:3] = torch.tensor(ends)
        lam[3] = float("nan")
        c["lam"] = lam
        kw = dict(scale=scale, initial_state=c["init"], seq_idx=c["seq"])
        y, st = ssd.gated_scan(c["x"], c["gates"], lam, return_states=True, **kw)
        grads = [ssd.gated_scan_bwd(c["x"], c["gates"], lam, c["dy"], d_final=c["dfin"], states=s,
                                    **kw) for s in (st, None)]
        torch.cuda.synchronize()
        n = _np(c)
        x, i, dy = n["x"][..., :3], n["gates"][..., 6:9], n["dy"][..., :3].copy()
        s = 1 / (1 + np.exp(-i))
        # a sigmoid off by 14 of 2^-24, one minus it by as much absolutely
        _close(y[..., :3], s * x, (2.0 ** -19 + HALF[io]) * np.abs(s * x) + TINY, "y")
        dy[:, -1] += n["dfin"][:, :3]
        for g in grads:
            assert not bool(g["dgates"][..., :3].any()), "dr"
            assert not bool(g["dlam"][:3].any()) and not bool(g["d_init"][:, :3].any())
            o = dy * s
            _close(g["dx"][..., :3], o, (2.0 ** -19 + HALF[io]) * np.abs(o) + TINY, "dx")
            o = dy * s * (1 - s) * x
            _close(g["dgates"][..., 6:9], o, 2.0 ** -19 * np.abs(dy * s * x) + HALF[io] * np.abs(o)
                   + TINY, "di")
            assert bool(torch.isnan(g["dx"][..., 3]).all()) and bool(torch.isnan(g["dlam"][3]))
            if scale == 8.0:
                for v in (g["dx"], g["dgates"][..., :6], g["dgates"][..., 6:], g["d_init"], g["dlam"]):
                    assert bool(torch.isfinite(v[..., 4:]).all())
    c = _case(6300, 2, l, 4, io, lam=(-3.0, 0.0))
    c["lam"] = torch.tensor([-3.0, 0.0, 1e38, np.inf], device="cuda")
    kw = dict(scale=0.0, initial_state=c["init"])
    y, fin = ssd.gated_scan(c["x"], c["gates"], c["lam"], return_final_state=True, **kw)
    g = ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], **kw)
    state = c["init"].clone()
    ssd.gated_step(state, c["x"][:, 0].contiguous(), c["gates"][:, 0].contiguous(), c["lam"], scale=0.0)
    torch.cuda.synchronize()
    assert torch.equal(fin, c["init"]) and torch.equal(state, c["init"])
    assert not bool(g["dx"].any()) and not bool(g["dgates"].any())
