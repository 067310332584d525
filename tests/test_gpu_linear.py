"""GPU parity of ssd_linear and ssd_linear_bwd (through the binding) against
the fp64 oracle in oracle/linear.py.

Tolerances, per element.  A product of K terms in fp32 is off by at most
K 2^-24 sum |a b| (each addition rounds once; MFMA sums in another order, the
bound holds for any).  The activation's first derivative is below 1.13 and its
own evaluation is off by at most 2^-20 (1 + |v|) (hardware exponential and
reciprocal, the error function).  An output in bf16 adds half a step, 2^-8 of
its value; fp32 2^-24.  The gradient at the pre-activation, e, is rounded to
bf16 before the products where an activation comes with it: 2^-8 |e| per term.
"""
import numpy as np
import pytest

from gpu_util import dev_tensor, log, to_f64, torch_mod

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _rand(seed, io, *shape, std=1.0):
    torch = torch_mod()
    a = (np.random.default_rng(seed).normal(size=shape) * std).astype(np.float32)
    t = torch.from_numpy(a).to("cuda")
    return t.to(torch.bfloat16) if io == "bf16" else t


def _guarded(shape, io):
    """An output between two runs of sentinels, and the check of both."""
    torch = torch_mod()
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    n = int(np.prod(shape))
    buf = torch.full((n + 8192,), 77.0, dtype=dt, device="cuda")
    out = buf[4096:4096 + n].view(shape)

    def check():
        assert bool((buf[:4096] == 77).all()) and bool((buf[4096 + n:] == 77).all())
    return out, check


def _close(g, o, tol, what):
    g = to_f64(g)
    assert g.shape == o.shape, (what, g.shape, o.shape)
    assert np.isfinite(g).all(), what
    err = np.abs(g - o) - tol
    assert (err <= 0).all(), "%s: worst excess %.3g at %s (got %r, want %r)" % (
        what, err.max(), np.unravel_index(err.argmax(), err.shape), g.flat[err.argmax()],
        o.flat[err.argmax()])


def _linear(m, k, n, io, act="none", bias=True, residual=True, pre=False, seed=0):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import linear as lo
    torch = torch_mod()
    x, w = _rand(seed, io, m, k), _rand(seed + 1, io, n, k, std=k ** -0.5)
    b = _rand(seed + 2, "f32", n) if bias else None
    r = _rand(seed + 3, io, m, n) if residual else None
    out, guard = _guarded((m, n), io)
    pout, pguard = _guarded((m, n), io)
    log("linear", m, k, n, io, act)
    got = ssd.linear(x, w, bias=b, activation=act, residual=r, return_pre=pre, out=out,
                     pre_out=pout if pre else None)
    torch.cuda.synchronize()
    guard()
    pguard()
    xo, wo = to_f64(x), to_f64(w)
    o, p = lo.linear(xo, wo, None if b is None else to_f64(b), act,
                     None if r is None else to_f64(r))
    acc = (k + 4) * 2.0 ** -24 * (np.abs(xo) @ np.abs(wo).T + (0 if b is None else 1) * 4)
    ev = 0 if act == "none" else 2.0 ** -20 * (1 + np.abs(p))
    tol = (1.13 * acc + ev) * 1.01 + HALF[io] * 1.01 * np.abs(o) + 2.0 ** -23 * np.abs(o)
    _close(got[0] if pre else got, o, tol, "out")
    if pre:
        _close(got[1], p, acc * 1.01 + HALF[io] * 1.01 * np.abs(p), "pre")
    return x, w, b, r


# one token and a few, the tile edges, ragged everything, odd widths, long contractions
SHAPES = [
    (1, 64, 16), (1, 2560, 512), (1, 33, 7), (1, 5120, 24), (2, 130, 1), (3, 100, 130),
    (5, 768, 3352), (7, 1, 5), (15, 1000, 100), (16, 2560, 96), (17, 96, 33), (31, 1536, 80),
    (33, 72, 64), (64, 640, 200), (65, 65, 65), (100, 2048, 64), (127, 128, 129), (128, 4096, 128),
    (129, 136, 257), (255, 768, 255), (256, 5120, 256), (300, 520, 260), (513, 31, 1027),
    (1000, 768, 1552), (2050, 200, 16), (4096, 64, 24), (1, 20000, 40), (300, 8, 4),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(shape, io):
    k = SHAPES.index(shape)
    act = ["none", "silu", "gelu", "sigmoid"][k % 4]
    _linear(*shape, io=io, act=act, bias=k % 3 != 0, residual=k % 2 == 0, pre=k % 4 != 0,
            seed=100 + 10 * k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
def test_linear_activations_over_their_range(act, io):
    """Pre-activations from -200 to 200: nothing overflows to NaN."""
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import linear as lo
    torch = torch_mod()
    v = np.concatenate([np.linspace(-12, 12, 481), [-200, -100, -50, 50, 100, 200, 0]])
    x = dev_tensor(v[:, None].astype(np.float32))
    x = x.to(torch.bfloat16) if io == "bf16" else x
    x = torch.cat([x, torch.zeros((x.shape[0], 15), dtype=x.dtype, device="cuda")], 1).contiguous()
    w = torch.zeros((4, 16), dtype=x.dtype, device="cuda")
    w[:, 0] = 1
    y = ssd.linear(x, w, activation=act)
    torch.cuda.synchronize()
    o, _ = lo.linear(to_f64(x), to_f64(w), None, act)
    _close(y, o, 2.0 ** -20 * (1 + np.abs(o)) + HALF[io] * np.abs(o), act)


def test_linear_residual_in_place_and_leading_axes():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    x, w = _rand(1, "bf16", 2, 37, 128), _rand(2, "bf16", 72, 128, std=0.1)
    r = _rand(3, "bf16", 2, 37, 72)
    want = ssd.linear(x, w, residual=r)
    keep = r.clone()
    got = ssd.linear(x, w, residual=keep, out=keep)
    torch.cuda.synchronize()
    assert got.data_ptr() == keep.data_ptr() and torch.equal(got, want)
    assert ssd.linear(x[:, :0].contiguous(), w).shape == (2, 0, 72)


def test_linear_nan_rows_stay_in_their_row():
    """A row with infinities or NaN reaches its own outputs only, also past a ragged edge."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for m in (3, 20, 130, 300):
        x, w = _rand(5, "bf16", m, 72), _rand(6, "bf16", 40, 72)
        want = ssd.linear(x, w)
        x[m - 1] = float("nan")
        x[m // 2] = float("inf")
        got = ssd.linear(x, w)
        torch.cuda.synchronize()
        rows = [i for i in range(m) if i not in (m - 1, m // 2)]
        assert torch.equal(got[rows], want[rows])
        assert bool(torch.isnan(got[m - 1]).all()) and not bool(torch.isfinite(got[m // 2]).any())


BWD = [(1, 64, 16), (1, 33, 7), (3, 1, 5), (5, 100, 130), (64, 128, 64), (65, 72, 80),
       (200, 770, 39), (128, 256, 128), (300, 264, 520), (1025, 96, 257), (2047, 130, 71),
       (4099, 64, 48), (1, 2560, 768), (17, 8, 4),
       (2, 4761, 300), (7, 80, 1000), (8, 513, 260), (4, 1024, 2047), (9, 72, 40), (8, 520, 9000),
       (1, 2561, 2000), (2, 8200, 555), (3, 4761, 1111), (6, 1031, 4444)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", BWD, ids=str)
def test_linear_bwd(shape, io):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import linear as lo
    torch = torch_mod()
    m, k, n = shape
    j = BWD.index(shape)
    act = ["gelu", "none", "silu", "sigmoid"][j % 4]
    seed = 1000 + 10 * j
    x, w = _rand(seed, io, m, k), _rand(seed + 1, io, n, k, std=n ** -0.5)
    dy, pre = _rand(seed + 2, io, m, n), _rand(seed + 3, io, m, n, std=2.0)
    log("linear_bwd", m, k, n, io, act)
    g = ssd.linear_bwd(dy, x, w, pre=None if act == "none" else pre, activation=act, bias=True)
    torch.cuda.synchronize()
    xo, wo, eo = to_f64(x), to_f64(w), to_f64(dy)
    r = lo.linear_grad(eo, xo, wo, to_f64(pre), act)
    # e: its evaluation, and for the products its rounding to the io type
    ea = np.abs(r["e"])
    ev = 0 if act == "none" else 2.0 ** -20 * np.abs(eo) * (1 + np.abs(to_f64(pre)))
    er = ev + (HALF[io] if act != "none" else 0) * ea
    mags = {"dx": (er @ np.abs(wo), ea @ np.abs(wo), n), "dweight": (er.T @ np.abs(xo),
                                                                    ea.T @ np.abs(xo), m)}
    for key, (by_e, mag, terms) in mags.items():
        o = r[key]
        _close(g[key], o, 1.01 * (by_e + (terms + 4) * 2.0 ** -24 * mag + HALF[io] * np.abs(o)), key)
    _close(g["dbias"], r["dbias"],
           (np.broadcast_to(ev, ea.shape).sum(0) + (m + 4) * 2.0 ** -24 * ea.sum(0)) * 1.01 + 1e-30,
           "dbias")


def test_linear_is_deterministic_and_sees_only_its_inputs():
    """The same call twice, the second on a workspace full of NaN, gives the same bits."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for m, k, n in ((1, 2560, 512), (200, 4096, 130), (256, 777, 255)):
        x, w = _rand(11, "bf16", m, k), _rand(12, "bf16", n, k, std=0.05)
        dy, pre = _rand(13, "bf16", m, n), _rand(14, "bf16", m, n)
        nb = max(ssd.linear_workspace_bytes(m, k, n), 256)
        nbb = ssd.linear_bwd_workspace_bytes(m, k, n, "gelu")
        outs = []
        for fill in (0, 255):
            ws = torch.full((nb,), fill, dtype=torch.uint8, device="cuda")
            wsb = torch.full((nbb,), fill, dtype=torch.uint8, device="cuda")
            y = ssd.linear(x, w, activation="silu", workspace=ws)
            g = ssd.linear_bwd(dy, x, w, pre=pre, activation="gelu", bias=True, workspace=wsb)
            outs.append([y, g["dx"], g["dweight"], g["dbias"]])
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_linear_on_another_stream():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    x, w = _rand(21, "bf16", 300, 512), _rand(22, "bf16", 260, 512, std=0.05)
    want = ssd.linear(x, w, activation="gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ssd.linear(x, w, activation="gelu")
    s.synchronize()
    assert torch.equal(got, want)


def test_linear_zero_rows_gradient():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    w = _rand(31, "bf16", 24, 40)
    e = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    g = ssd.linear_bwd(e, torch.empty((0, 40), dtype=torch.bfloat16, device="cuda"), w, bias=True)
    torch.cuda.synchronize()
    assert g["dx"].shape == (0, 40)
    assert not bool(g["dweight"].any()) and not bool(g["dbias"].any())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_linear_of_row_slices(io):
    """Runs of rows of larger tensors, at every width's own alignment."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for m, k, n in ((3, 33, 7), (20, 72, 36), (150, 36, 33)):
        x, w, r = (_rand(41 + j, io, s0 + 1, s1)[1:] for j, (s0, s1) in
                   enumerate(((m, k), (n, k), (m, n))))
        b = _rand(44, "f32", n + 1)[1:]
        got = ssd.linear(x, w, bias=b, residual=r, activation="silu")
        want = ssd.linear(x.clone(), w.clone(), bias=b.clone(), residual=r.clone(),
                          activation="silu")
        gg = ssd.linear_bwd(r, x, w, pre=r, activation="gelu", bias=True)
        gw = ssd.linear_bwd(r.clone(), x.clone(), w.clone(), pre=r.clone(), activation="gelu",
                            bias=True)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for key in gg:
            assert torch.equal(gg[key], gw[key]), key


def test_offsets_beyond_32_bits():
    """An output of 2.9e9 values: sampled rows, and the weight's gradient over all
    of them, against fp64 (tolerances as above)."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    m, k, n = 700001, 24, 4096
    log("linear", m, k, n)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((m, k), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((n, k), generator=gen, device="cuda", dtype=torch.bfloat16)
    y = ssd.linear(x, w)
    g = ssd.linear_bwd(y, x, w, bias=True)
    torch.cuda.synchronize()
    rows = [0, 1, 127, 128, 350000, 524287, 524288, m - 130, m - 2, m - 1]
    xo, wo = to_f64(x[rows]), to_f64(w)
    o, mag = xo @ wo.T, np.abs(xo) @ np.abs(wo).T
    _close(y[rows], o, 1.01 * (HALF["bf16"] * np.abs(o) + (k + 4) * 2.0 ** -24 * mag), "y")
    e = to_f64(y[rows])
    o, mag = e @ wo, np.abs(e) @ np.abs(wo)
    _close(g["dx"][rows], o, 1.01 * (HALF["bf16"] * np.abs(o) + (n + 4) * 2.0 ** -24 * mag), "dx")
    dw = torch.zeros((n, k), dtype=torch.float64, device="cuda")
    ma, db, mb = torch.zeros_like(dw), torch.zeros(n, dtype=torch.float64, device="cuda"), 0
    for i in range(0, m, 50000):
        ec, xc = y[i:i + 50000].double().t().contiguous(), x[i:i + 50000].double()
        dw += ec @ xc
        ma += ec.abs() @ xc.abs()
        db += ec.sum(1)
        mb = mb + ec.abs().sum(1)
    o = to_f64(g["dweight"])
    tol = 1.01 * (HALF["bf16"] * dw.abs() + (m + 4) * 2.0 ** -24 * ma).cpu().numpy()
    assert (np.abs(o - dw.cpu().numpy()) <= tol).all()
    tol = 1.01 * ((m + 4) * 2.0 ** -24 * mb).cpu().numpy()
    assert (np.abs(to_f64(g["dbias"]) - db.cpu().numpy()) <= tol).all()
