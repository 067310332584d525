"""GPU parity of ssd_gated_scan, ssd_gated_scan_bwd and ssd_gated_step (through
the binding) against the fp64 oracle in oracle/gated.py.

Tolerances, per element.  In fp32 a decay is off by at most about 26 2^-24 of
itself (the gate's sigmoid: 14 with the argument of its exponential at most 8;
the rate: softplus and two products, 24 in all on u, which scales a's error by
u <= 1; the exponential 2) and an added value by at most 32 2^-24 (half the
error of u and of the series in beta, the gate's 14, the square root and three
products); both are covered by delta = 2^-18, also with the roundings of the
maps' composition (one per token and map).  The oracle carries delta through
the recurrence and the gradient to first order.  An output in bf16 adds half a
step, 2^-8 of its value.
"""
import numpy as np
import pytest

from gpu_util import log, to_f64, torch_mod

pytestmark = pytest.mark.gpu

DELTA = 2.0 ** -18
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _case(seed, b, l, d, io, docs=False, init=True):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32

    def t(*shape, std=1.0):
        return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).to("cuda")
    a = 0.9 + 0.0995 * rng.random(d)
    lam = torch.from_numpy(np.log(np.expm1(-np.log(a) / 8.0)).astype(np.float32)).to("cuda")
    seq = None
    if docs:
        seq = torch.from_numpy(np.cumsum(rng.random((b, l)) < 0.05, 1).astype(np.int32)).to("cuda")
    return dict(x=t(b, l, d).to(dt), gates=t(b, l, 2 * d).to(dt), lam=lam,
                init=t(b, d) if init else None, seq=seq, dy=t(b, l, d).to(dt), dfin=t(b, d))


def _np(c):
    return {k: None if v is None else (v.cpu().numpy() if k == "seq" else to_f64(v))
            for k, v in c.items()}


def _close(g, o, tol, what):
    g = to_f64(g)
    assert g.shape == o.shape, (what, g.shape, o.shape)
    assert np.isfinite(g).all(), what
    err = np.abs(g - o) - tol
    assert (err <= 0).all(), "%s: worst excess %.3g at %s (got %r, want %r)" % (
        what, err.max(), np.unravel_index(err.argmax(), err.shape), g.flat[err.argmax()],
        o.flat[err.argmax()])


# (batch, seqlen, dim): one token, tile edges, many tiles, every lane width
SHAPES = [(1, 1, 1), (2, 1, 8), (3, 7, 5), (1, 63, 64), (2, 64, 130), (2, 65, 256), (1, 127, 257),
          (1, 128, 260), (2, 200, 771), (4, 513, 34), (1, 1000, 515), (1, 4100, 20), (2, 2048, 512),
          (3, 1001, 77), (1, 20000, 4)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_scan(shape, io):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import gated as go
    torch = torch_mod()
    k = SHAPES.index(shape)
    c = _case(2000 + k, *shape, io=io, docs=k % 3 == 0, init=k % 2 == 0)
    log("gated_scan", shape, io)
    y, fin, st = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"],
                                seq_idx=c["seq"], return_final_state=True, return_states=True)
    torch.cuda.synchronize()
    n = _np(c)
    r = go.scan(n["x"], n["gates"], n["lam"], 8.0, n["init"], n["seq"], delta=DELTA)
    _close(y, r["y"], r["err"] + HALF[io] * np.abs(r["y"]) * 1.01 + 1e-30, "y")
    _close(fin, r["final"], r["err"][:, -1] + 2.0 ** -24 * np.abs(r["final"]), "final")
    at = [min(64 * (j + 1), shape[1]) - 1 for j in range(-(-shape[1] // 64))]
    _close(st, r["states"], r["err"][:, at] + 2.0 ** -24 * np.abs(r["states"]), "states")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_scan_bwd(shape, io):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import gated as go
    torch = torch_mod()
    k = SHAPES.index(shape)
    c = _case(3000 + k, *shape, io=io, docs=k % 3 == 1, init=k % 2 == 1)
    dfin = c["dfin"] if k % 4 < 2 else None
    log("gated_scan_bwd", shape, io)
    _, st = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"],
                           seq_idx=c["seq"], return_states=True)
    runs = [ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], initial_state=c["init"],
                               d_final=dfin, seq_idx=c["seq"], states=s) for s in (None, st)]
    torch.cuda.synchronize()
    n = _np(c)
    r = go.grad(n["x"], n["gates"], n["lam"], 8.0, n["dy"], n["init"], n["seq"],
                None if dfin is None else n["dfin"], delta=DELTA)
    for g in runs:
        for key in ("dx", "dgates"):
            _close(g[key], r[key], r["err_" + key] + HALF[io] * np.abs(r[key]) * 1.01 + 1e-30, key)
        _close(g["dlam"], r["dlam"], r["err_dlam"] + 1e-30, "dlam")
        assert ("d_init" in g) == (c["init"] is not None)
        if "d_init" in g:
            _close(g["d_init"], r["d_init"], r["err_d_init"] + 2.0 ** -23 * np.abs(r["d_init"]),
                   "d_init")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 2560), (3, 5), (7, 130), (256, 512)], ids=str)
def test_gated_step_continues_the_scan(shape, io):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import gated as go
    torch = torch_mod()
    b, d = shape
    c = _case(4000 + b + d, b, 6, d, io=io)
    _, state = ssd.gated_scan(c["x"][:, :2].contiguous(), c["gates"][:, :2].contiguous(), c["lam"],
                              initial_state=c["init"], return_final_state=True)
    log("gated_step", shape, io)
    n = _np(c)
    r = go.scan(n["x"], n["gates"], n["lam"], 8.0, n["init"], delta=DELTA)
    for t in range(2, 6):
        y = ssd.gated_step(state, c["x"][:, t].contiguous(), c["gates"][:, t].contiguous(),
                           c["lam"])
        torch.cuda.synchronize()
        o, e = r["y"][:, t], r["err"][:, t]
        _close(y, o, e + HALF[io] * 1.01 * np.abs(o), "y")
        _close(state, o, e + 2.0 ** -24 * np.abs(o), "state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gates_shut_and_open(io):
    """Gates at the ends of their range: a decay of one (nothing added, zero
    gradients, no NaN) and the strongest decay, and lam far out on both sides."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    b, l, d = 2, 130, 24
    c = _case(5000, b, l, d, io=io)
    g = torch.empty_like(c["gates"])
    g[..., :8], g[..., 8:16], g[..., 16:d] = -1e4, -90.0, 1e4
    g[..., d:] = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1e4, -1e4)
    lam = c["lam"].clone()
    lam[3::8], lam[5::8], lam[6::8] = -200.0, 60.0, -95.0
    y, fin = ssd.gated_scan(c["x"], g, lam, initial_state=c["init"], return_final_state=True)
    gr = ssd.gated_scan_bwd(c["x"], g, lam, c["dy"], initial_state=c["init"], d_final=c["dfin"])
    torch.cuda.synchronize()
    for t in (y, fin, *gr.values()):
        assert bool(torch.isfinite(t).all())
    # shut: the state stays the initial one, bit for bit
    assert torch.equal(fin[:, :8], c["init"][:, :8])
    assert torch.equal(y[:, :, :8], c["init"][:, None, :8].to(y.dtype).expand(b, l, 8))
    assert not bool(gr["dx"][..., :8].any()) and not bool(gr["dgates"][..., :8].any())


def test_final_state_in_place_and_empty_sequence():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for l in (5, 200):
        c = _case(5100 + l, 2, l, 36, io="bf16")
        _, want = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"],
                                 return_final_state=True)
        h = c["init"].clone()
        y, got = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=h,
                                return_final_state=True, final_out=h)
        torch.cuda.synchronize()
        assert got.data_ptr() == h.data_ptr() and torch.equal(got, want)
    for init in (None, c["init"]):
        y, fin = ssd.gated_scan(c["x"][:, :0].contiguous(), c["gates"][:, :0].contiguous(),
                                c["lam"], initial_state=init, return_final_state=True)
        torch.cuda.synchronize()
        assert y.shape == (2, 0, 36)
        assert torch.equal(fin, torch.zeros_like(fin) if init is None else init)


@pytest.mark.parametrize("l", [40, 1000])
def test_scan_reads_no_stale_workspace_and_repeats(l):
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = _case(5200, 2, l, 260, io="bf16", docs=True)
    outs = []
    for fill in (0, 255, 0x7f):
        ws = torch.full((ssd.gated_scan_workspace_bytes(2, l, 260) + 256,), fill,
                        dtype=torch.uint8, device="cuda")
        wb = torch.full((ssd.gated_scan_bwd_workspace_bytes(2, l, 260) + 256,), fill,
                        dtype=torch.uint8, device="cuda")
        r = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"],
                           seq_idx=c["seq"], return_final_state=True, return_states=True,
                           workspace=ws)
        g = ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], initial_state=c["init"],
                               seq_idx=c["seq"], workspace=wb)
        outs.append(list(r) + [g[k] for k in sorted(g)])
    torch.cuda.synchronize()
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


def test_channels_and_rows_do_not_mix():
    """A NaN in one channel of one sequence stays there; guards around every output hold."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    b, l, d = 3, 150, 70
    c = _case(5300, b, l, d, io="bf16")
    want = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"])
    x = c["x"].clone()
    x[1, 20, 33] = float("nan")
    buf = torch.full((b * l * d + 2048,), 5.0, dtype=x.dtype, device="cuda")
    out = buf[1024:1024 + b * l * d].view(b, l, d)
    ssd.gated_scan(x, c["gates"], c["lam"], initial_state=c["init"], out=out)
    torch.cuda.synchronize()
    bad = torch.isnan(out)
    assert bool(bad[1, 20:, 33].all())
    bad[1, 20:, 33] = False
    assert not bool(bad.any())
    keep = torch.ones_like(bad)
    keep[1, 20:, 33] = False
    assert torch.equal(out[keep], want[keep])
    assert bool((buf[:1024] == 5).all()) and bool((buf[1024 + b * l * d:] == 5).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_tensors_at_odd_offsets(io):
    """Views that start off every vector width give the same bits as aligned copies."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = _case(5400, 1, 301, 64, io=io)

    def off(t, by):
        buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        v = buf[by:].view(t.shape)
        v.copy_(t)
        return v
    for by in (1, 2):
        o = {k: off(c[k], by) for k in ("x", "gates", "lam", "init", "dy", "dfin")}
        a = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"],
                           return_final_state=True)
        b = ssd.gated_scan(o["x"], o["gates"], o["lam"], initial_state=o["init"],
                           return_final_state=True)
        ga = ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], initial_state=c["init"],
                                d_final=c["dfin"])
        gb = ssd.gated_scan_bwd(o["x"], o["gates"], o["lam"], o["dy"], initial_state=o["init"],
                                d_final=o["dfin"])
        h = off(c["init"], by)
        y = ssd.gated_step(h, o["x"][:, 1], o["gates"][:, 1], o["lam"])
        h2 = c["init"].clone()
        y2 = ssd.gated_step(h2, c["x"][:, 1], c["gates"][:, 1], c["lam"])
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(h, h2)
        for u, v in zip(a, b):
            assert torch.equal(u, v)
        for k in ga:
            assert torch.equal(ga[k], gb[k]), k


def test_every_token_its_own_document():
    """With a new document at every token the state is what the token adds, and
    no gradient crosses."""
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import gated as go
    torch = torch_mod()
    c = _case(5500, 2, 300, 40, io="f32")
    seq = torch.arange(300, dtype=torch.int32, device="cuda").repeat(2, 1)
    y, fin = ssd.gated_scan(c["x"], c["gates"], c["lam"], seq_idx=seq, return_final_state=True)
    g = ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], seq_idx=seq)
    torch.cuda.synchronize()
    n = _np(c)
    r = go.scan(n["x"], n["gates"], n["lam"], 8.0, None, seq.cpu().numpy(), delta=DELTA)
    _close(y, r["y"], r["err"] + 1e-30, "y")
    assert torch.equal(fin, y[:, -1])
    k = go.grad(n["x"], n["gates"], n["lam"], 8.0, n["dy"], None, seq.cpu().numpy(), None,
                delta=DELTA)
    for key in ("dx", "dgates", "dlam"):
        _close(g[key], k[key], k["err_" + key] + 1e-30, key)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, give what each gives alone."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    cs = [_case(5600 + k, 2, 3000, 512, io="bf16", docs=k == 1) for k in range(2)]

    def run(c):
        y, fin, st = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"],
                                    seq_idx=c["seq"], return_final_state=True,
                                    return_states=True)
        g = ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], initial_state=c["init"],
                               seq_idx=c["seq"], d_final=c["dfin"])
        return [y, fin, st] + [g[k] for k in sorted(g)]
    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = run(cs[k])
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(got[k], want[k]):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """Gates of 2.4e9 values (4.9 GB): the last tokens equal a scan of the tail
    from the state kept before it, up to the rounding of the states on the way
    (a few 2^-24) and one bf16 step."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    b, l, d = 1, 300032, 4096
    log("gated_scan", b, l, d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((b, l, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    gates = torch.randn((b, l, 2 * d), generator=gen, device="cuda", dtype=torch.bfloat16)
    lam = torch.full((d,), -6.0, device="cuda")
    y, fin, st = ssd.gated_scan(x, gates, lam, return_final_state=True, return_states=True)
    at = l - 512
    yt, ft = ssd.gated_scan(x[:, at:].clone(), gates[:, at:].clone(), lam,
                            initial_state=st[:, at // 64 - 1].clone(), return_final_state=True)
    torch.cuda.synchronize()
    a, o = to_f64(y[:, at:]), to_f64(yt)
    assert (np.abs(a - o) <= 2.0 ** -7 * np.abs(o) + 1e-5).all()
    np.testing.assert_allclose(to_f64(fin), to_f64(ft), rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [33, 128])
def test_documents_do_not_reach_each_other(d, io):
    """Infinities and NaN in some documents (and in the state that the first one
    starts from) leave the bits of the others as they are, and every later token
    of their own document not finite."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    b, l = 2, 2300
    c = _case(29, b, l, d, io)
    # starts at the edges of waves, tiles and groups, inside them, and alone
    starts = [0, 1, 63, 64, 65, 128, 250, 256, 263, 511, 512, 1024, 1025, 1536, 1700, 2048, 2299]
    seq = torch.zeros(l, dtype=torch.int32)
    for k, t in enumerate(starts):
        seq[t:] = k
    seq = seq.repeat(b, 1).cuda()

    def run(c):
        y, fin, st = ssd.gated_scan(c["x"], c["gates"], c["lam"], initial_state=c["init"], seq_idx=seq,
                                    return_final_state=True, return_states=True)
        for s in (st, None):
            g = ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], initial_state=c["init"],
                                   seq_idx=seq, d_final=c["dfin"], states=s)
            yield y, fin, g["dx"], g["dgates"]

    clean = list(run(c))
    for odd in (0, 1):
        bad = (seq[0] % 2 == odd)
        p = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
        first = [t for k, t in enumerate(starts) if k % 2 == odd]
        last = [t - 1 for k, t in enumerate(starts) if k and (k - 1) % 2 == odd]
        p["x"][:, first] = float("nan")
        p["x"][:, last] = float("inf")
        p["dy"][:, last] = float("nan")
        p["gates"][:, first[1:], :d // 2] = float("nan")
        if odd == 0:
            p["init"][:] = float("inf")  # the first document's; the last is even too
            p["dfin"][:] = float("nan")
        for (y, fin, dx, dg), (y0, fin0, dx0, dg0) in zip(run(p), clean):
            for g, w in ((y, y0), (dx, dx0), (dg, dg0)):
                assert torch.equal(g[:, ~bad], w[:, ~bad])
            assert not torch.isfinite(y[:, bad]).any()
            assert not torch.isfinite(fin).any() if odd == 0 else torch.equal(fin, fin0)
            starting = torch.tensor(first)
            assert torch.isnan(dx[:, starting]).all()


@pytest.mark.parametrize("l", [1, 40, 300])
def test_rates_at_their_ends(l):
    """A rate of exactly zero (lam = -inf, or far below) keeps the state and shuts
    the input, one without bound (lam = inf) keeps nothing; a NaN stays in its
    channel."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = _case(31, 2, l, 6, "f32")
    lam = torch.tensor([-float("inf"), -1e4, float("inf"), 1e4, float("nan"), -3.0], device="cuda")
    kw = dict(initial_state=c["init"])
    y, fin, st = ssd.gated_scan(c["x"], c["gates"], lam, return_final_state=True,
                                return_states=True, **kw)
    g = ssd.gated_scan_bwd(c["x"], c["gates"], lam, c["dy"], states=st, **kw)
    state = c["init"].clone()
    y1 = ssd.gated_step(state, c["x"][:, 0].contiguous(), c["gates"][:, 0].contiguous(), lam)
    for t in (y, y1[:, None]):
        assert torch.equal(t[..., :2], c["init"][:, None, :2].expand_as(t[..., :2]))
        assert torch.isnan(t[..., 4]).all() and torch.isfinite(t[..., 5]).all()
    assert torch.equal(g["dgates"][..., :2], torch.zeros_like(g["dgates"][..., :2]))
    assert torch.equal(g["dx"][..., :2], torch.zeros_like(g["dx"][..., :2]))
    # a = 0, beta = 1: sigmoid(i) x, off by at most 14 2^-24 and a rounding
    want = torch.sigmoid(c["gates"][..., 8:10].double()) * c["x"][..., 2:4].double()
    assert ((y[..., 2:4] - want).abs() <= 2.0 ** -20 * want.abs()).all()
    assert torch.isnan(g["dx"][..., 4]).all() and torch.isfinite(g["dx"][..., 5]).all()
