"""The gated delta rule's kernels (scan, gradient, step) against the fp64 oracle."""
import numpy as np
import pytest

from delta_util import BOUNDS, as64, delta_case, io_dtype, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "dt", "A", "beta")


def _scan(c, **kw):
    import mamba_ssd_chunked_chunk_amd as ssd
    return ssd.delta_scan(*(c[k] for k in NAMES), dt_bias=c["dt_bias"], initial_state=c["init"],
                          seq_idx=c["seq"], **kw)


def _bwd(c, states=None, **kw):
    import mamba_ssd_chunked_chunk_amd as ssd
    return ssd.delta_scan_bwd(*(c[k] for k in NAMES), c["dy"], dt_bias=c["dt_bias"],
                              initial_state=c["init"], seq_idx=c["seq"], d_final=c["d_final"],
                              states=states, **kw)


def _o(c):
    e = as64(c)
    e.pop("dy"), e.pop("d_final")
    return e


def check_scan(c, io, what, **kw):
    y, fin, st = _scan(c, return_final_state=True, return_states=True, **kw)
    ref = oracle.scan(**_o(c), **kw)
    for name, x, o, bound in (("y", y, ref["y"], "y"), ("final", fin, ref["final"], "state"),
                              ("states", st, ref["states"], "state")):
        r = rel(x, o)
        log(what, name, "%.2e" % r)
        assert r <= BOUNDS[io][bound], (what, name, r)
        if o.size:  # no single element is far off either
            worst = np.abs(x.double().cpu().numpy() - o) / (np.abs(o) + np.sqrt(np.mean(o * o)) + 1e-300)
            assert worst.max() <= 16 * BOUNDS[io][bound], (what, name, worst.max())
    return st


def check_bwd(c, io, what, states=None, **kw):
    got = _bwd(c, states, **kw)
    e = as64(c)
    ref = oracle.grad(**_o(c), dy=e["dy"], d_final=e["d_final"], **kw)
    assert set(got) == set(ref)
    for name, o in ref.items():
        r = rel(got[name], o)
        log(what, name, "%.2e" % r)
        assert r <= BOUNDS[io][name], (what, name, r)
    return got


SHAPES = [  # b, l, h, g, n, p
    (2, 1, 3, 3, 32, 16),
    (1, 2, 2, 1, 64, 64),
    (2, 63, 4, 2, 128, 128),
    (1, 64, 4, 4, 128, 64),
    (2, 65, 6, 2, 64, 32),
    (1, 130, 4, 1, 32, 128),
    (3, 200, 2, 2, 128, 16),
    (1, 333, 8, 2, 64, 64),
    (2, 257, 3, 1, 128, 32),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("norm,packed,init", [(False, False, False), (True, True, True)],
                         ids=["plain", "norm-packed-init"])
def test_scan_and_gradient(shape, io, norm, packed, init):
    c = delta_case(sum(shape), *shape, io, normalize=norm, packed=packed, init=init)
    kw = dict(normalize=norm)
    st = check_scan(c, io, "scan", **kw)
    a = check_bwd(c, io, "gradient", states=st, **kw)
    b = check_bwd(c, io, "gradient, states again", **kw)
    # the forward pass keeps the states that the gradient would compute
    torch = torch_mod()
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_every_value_width_and_key_width(io):
    for n in (32, 64, 128):
        for p in (16, 32, 64, 128):
            c = delta_case(n + p, 2, 100, 2, 1, n, p, io, init=True)
            st = check_scan(c, io, "scan %d %d" % (n, p))
            check_bwd(c, io, "gradient %d %d" % (n, p), states=st)


# So many heads that the compute units are full with one wave per 16 columns, in
# workgroups of every size; the last two have more than one head of a group in a
# wave of the preparation.
MANY = [  # b, l, h, g, n, p
    (2, 130, 132, 4, 32, 16),
    (1, 65, 260, 130, 128, 16),
    (2, 200, 66, 6, 64, 32),
    (3, 70, 24, 8, 128, 64),
    (1, 129, 36, 36, 32, 128),
    (1, 66, 264, 88, 64, 128),
    (1, 65, 258, 3, 128, 128),
    (6, 130, 256, 128, 32, 16),
    (9, 250, 180, 60, 32, 16),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_many_heads(shape, io):
    c = delta_case(sum(shape), *shape, io, normalize=True, packed=True, init=True)
    kw = dict(normalize=True)
    st = check_scan(c, io, "scan", **kw)
    check_bwd(c, io, "gradient", states=st, **kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,p", [(32, 16), (64, 128), (128, 64), (128, 128)])
def test_steps_continue_a_scan(io, n, p):
    """Seventy steps from a scan's final state, each against the oracle from the
    same state; the step's arithmetic is fp32, its y rounded once."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = delta_case(7 + n + p, 2, 30, 4, 2, n, p, io, normalize=True)
    _, st = _scan(c, normalize=True, return_final_state=True)
    d = delta_case(8 + n + p, 2, 70, 4, 2, n, p, io, normalize=True)
    e = as64(d)
    for t in range(70):
        before = st.double().cpu().numpy()
        tok = [d[k] if k == "A" else d[k][:, t].contiguous() for k in NAMES]
        y = ssd.delta_step(st, *tok, dt_bias=d["dt_bias"], normalize=True)
        yo, so = oracle.step(before, *(e[k] if k == "A" else e[k][:, t] for k in NAMES),
                             dt_bias=e["dt_bias"], normalize=True)
        assert rel(st, so) < 1e-6 and rel(y, yo) < (2e-6 if io == "f32" else 2.0 ** -8), t
    # and the same tokens in one scan
    c2 = dict(d, init=_scan(c, normalize=True, return_final_state=True)[1])
    _, fin = _scan(c2, normalize=True, return_final_state=True)
    assert rel(fin, st.double().cpu().numpy()) < BOUNDS["f32"]["state"]
    assert torch.isfinite(fin).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_borders(io):
    """Decays that forget everything, none at all, beta of zero and two, rows of
    zeros in q and k, a clamp that is met on both sides, no bias and no softplus."""
    base = dict(b=2, l=150, h=4, g=2, n=64, p=32, io=io)
    torch = torch_mod()
    mk = lambda seed, **kw: delta_case(seed, **base, init=True, packed=True, **kw)  # noqa: E731

    def every(t, step, value):
        t = t.clone()
        t[:, ::step] = value
        return t
    cases = [
        ("strong decay", mk(1, A=lambda A: A * 1e6), {}),
        ("mixed decay", mk(2, dt=lambda t: every(t, 7, 60.0), A=lambda A: A * 20), {}),
        ("no decay", mk(3, A=lambda A: A * 0), {}),
        ("beta zero", mk(4, beta=lambda t: every(t, 3, 0.0)), {}),
        ("beta two", mk(5, beta=lambda t: every(t, 2, 2.0), k=lambda k: k * 0.99), {}),
        ("zero keys", mk(6, k=lambda k: every(k, 5, 0.0), q=lambda q: every(q, 4, 0.0)),
         dict(normalize=True)),
        ("zero keys, no eps", mk(7, k=lambda k: every(k, 5, 0.0), q=lambda q: every(q, 4, 0.0)),
         dict(normalize=True, norm_eps=0.0)),
        ("clamp", mk(8), dict(dt_limit=(0.02, 0.05))),
        ("raw steps", mk(9, dt=lambda t: t.abs() * 0.1, dt_bias=lambda t: None),
         dict(dt_softplus=False)),
        ("scale", mk(10), dict(scale=3.5)),
    ]
    for what, c, kw in cases:
        st = check_scan(c, io, what, **kw)
        check_bwd(c, io, what, states=st, **kw)
    c = mk(11, beta=lambda t: torch.zeros_like(t))
    assert torch.equal(_bwd(c)["dv"], torch.zeros_like(c["v"]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-18, 1e15])
def test_magnitudes(io, size):
    """Values, queries and cotangents far outside fp16's range (each operand has its
    own power of two); keys of any size where the call normalises them."""
    big = max(size, 1.0)  # with smaller keys norm_eps would outweigh them
    c = delta_case(20, 2, 130, 2, 1, 64, 32, io, normalize=True, init=True, v=lambda v: v * size,
                   k=lambda k: k * big, q=lambda q: q * big, dy=lambda t: t * size)
    c["init"] = c["init"] * size
    c["d_final"] = c["d_final"] * size
    check_scan(c, io, "size %g" % size, normalize=True)
    check_bwd(c, io, "size %g" % size, normalize=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("v,dy", [(1e-25, 1e6), (1e8, 1e-26), (1e-18, 1.0), (1e15, 1e12)])
def test_magnitudes_of_values_and_cotangents(io, v, dy):
    """Values and cotangents of different sizes, a group of 16 value columns of
    nothing but zeros beside one that is large, and one far below it."""
    c = delta_case(23, 2, 130, 2, 1, 64, 64, io, normalize=True, init=True, v=lambda t: t * v,
                   dy=lambda t: t * dy)
    c["init"], c["d_final"] = c["init"] * v, c["d_final"] * dy
    for name, axis in (("v", 3), ("dy", 3), ("init", 3), ("d_final", 3)):
        c[name].narrow(axis, 16, 16).zero_()
        c[name].narrow(axis, 48, 16).mul_(2.0 ** -40)
    check_scan(c, io, "sizes %g %g" % (v, dy), normalize=True)
    got = check_bwd(c, io, "sizes %g %g" % (v, dy), normalize=True)
    assert (got["dv"][..., 16:32] == 0).all() and (got["d_init"][..., 16:32] == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_repeated_keys(io):
    """One key over and over, and nearly one: the triangle's inverse is furthest
    from the identity.  Errors gather along the chunk: four times the bound."""
    for beta in (1.0, 0.5):
        c = delta_case(30, 1, 128, 2, 1, 32, 16, io, beta=lambda t: t * 0 + beta,
                       k=lambda k: k[:, :1].expand_as(k).contiguous(), A=lambda A: A * 0.01)
        got = _scan(c, return_final_state=True)
        ref = oracle.scan(**_o(c))
        assert rel(got[0], ref["y"]) <= 4 * BOUNDS[io]["y"]
        assert rel(got[1], ref["final"]) <= 4 * BOUNDS[io]["state"]


def test_final_state_in_place_and_out_arguments():
    torch = torch_mod()
    c = delta_case(40, 2, 100, 4, 2, 64, 64, "bf16", init=True)
    y, fin, st = _scan(c, return_final_state=True, return_states=True)
    own = dict(c, init=c["init"].clone())
    out = torch.full_like(y, 7.0)
    y2, fin2, st2 = _scan(own, return_final_state=True, return_states=True, out=out,
                          final_out=own["init"], states_out=torch.full_like(st, 7.0))
    assert y2 is out and fin2 is own["init"]
    assert torch.equal(y, y2) and torch.equal(fin, fin2) and torch.equal(st, st2)
    assert torch.equal(_scan(c), y)
    assert torch.equal(st[:, -1], fin)


def test_empty_calls():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = delta_case(41, 2, 0, 4, 2, 64, 64, "bf16", init=True)
    y, fin, st = _scan(c, return_final_state=True, return_states=True)
    assert y.shape == (2, 0, 4, 64) and st.shape == (2, 0, 4, 64, 64)
    assert torch.equal(fin, c["init"])
    c["init"] = None
    assert torch.equal(_scan(c, return_final_state=True)[1], torch.zeros_like(fin))
    with pytest.raises(ssd.SsdError):
        _bwd(c)
    c = delta_case(42, 0, 5, 4, 2, 64, 64, "f32")
    assert _scan(c).shape == (0, 5, 4, 64)


def test_workspace_contents_and_neighbours_do_not_matter():
    """Workspaces of NaN patterns give the same bits, and nothing is written behind
    the outputs or the workspace."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for io in ("bf16", "f32"):
        b, l, h, g, n, p = 2, 91, 4, 2, 64, 32
        c = delta_case(43, b, l, h, g, n, p, io, normalize=True, packed=True, init=True)

        def guarded(shape, dtype):
            size = int(np.prod(shape))
            flat = torch.full((size + 256,), 3.0, dtype=dtype, device="cuda")
            return flat, flat[:size].view(shape)
        want = _scan(c, normalize=True, return_final_state=True, return_states=True)
        fy, y = guarded((b, l, h, p), io_dtype(io))
        ff, f = guarded((b, h, n, p), torch.float32)
        fs, s = guarded((b, 2, h, n, p), torch.float32)
        for fill in (0, 255):
            need = ssd.delta_scan_workspace_bytes(b, l, h, p, n, g, io)
            ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
            _scan(c, normalize=True, return_final_state=True, return_states=True, out=y, final_out=f,
                  states_out=s, workspace=ws[:need])
            for x, o in zip((y, f, s), want):
                assert torch.equal(x, o)
            assert (ws[need:] == fill).all()
            for flat in (fy, ff, fs):
                assert (flat[-256:] == 3.0).all()
            for states in (None, s):
                need = ssd.delta_scan_bwd_workspace_bytes(b, l, h, p, n, g, io, states is not None)
                ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
                got = _bwd(c, states, normalize=True, workspace=ws[:need])
                ref = _bwd(c, states, normalize=True)
                for k in got:
                    assert torch.equal(got[k], ref[k]), (io, fill, k)
                assert (ws[need:] == fill).all()


def test_repeats_bit_for_bit():
    torch = torch_mod()
    c = delta_case(44, 4, 700, 16, 4, 128, 64, "bf16", normalize=True, packed=True)
    a, b = (_scan(c, normalize=True, return_final_state=True, return_states=True) for _ in range(2))
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    a, b = (_bwd(c, normalize=True) for _ in range(2))
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_two_calls_at_once_on_two_streams():
    torch = torch_mod()
    cases = [delta_case(50 + i, 2, 400, 8, 4, 128, 64, "bf16", normalize=True) for i in range(2)]
    want = [(_scan(c, normalize=True), _bwd(c, normalize=True)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i] = (_scan(c, normalize=True), _bwd(c, normalize=True))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0])
        for k in w[1]:
            assert torch.equal(g[1][k], w[1][k]), k


def test_graph_replays():
    """Scan, gradient and step captured together; every replay on new inputs against
    the eager calls, with eager work between the replays."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    shape = (2, 150, 4, 2, 64, 64, "bf16")
    c = delta_case(60, *shape, init=True)
    state = c["init"].clone()
    tok = lambda c: [c[k] if k == "A" else c[k][:, 0].contiguous() for k in NAMES]  # noqa: E731
    one = tok(c)

    def work():
        y, fin, st = _scan(c, return_final_state=True, return_states=True)
        g = _bwd(c, st)
        ys = ssd.delta_step(state, *one, dt_bias=c["dt_bias"])
        return [y, fin, st, ys] + [g[k] for k in sorted(g)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(3):
        new = delta_case(61 + i, *shape, init=True)
        for k, v in new.items():
            if v is not None:
                c[k].copy_(v)
        for x, v in zip(one, tok(new)):
            x.copy_(v)
        state.copy_(new["init"])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        state.copy_(new["init"])
        for x, o in zip(got, work()):
            assert torch.equal(x, o)


def test_offsets_beyond_32_bits():
    """v, y and the states beyond 4 GB: the last rows as a call of their own gives them."""
    torch = torch_mod()
    b, l, h, g, n, p = 9, 4096, 1024, 1, 32, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rnd = lambda *s, dtype=torch.bfloat16: torch.randn(s, generator=gen, device="cuda",  # noqa: E731
                                                       dtype=torch.float32).to(dtype)
    c = dict(q=rnd(b, l, g, n), k=rnd(b, l, g, n), dt=rnd(b, l, h), A=-rnd(h, dtype=torch.float32).abs(),
             beta=torch.rand((b, l, h), generator=gen, device="cuda").bfloat16(),
             dt_bias=rnd(h, dtype=torch.float32) - 3, init=None, seq=None)
    c["v"] = torch.empty((b, l, h, p), dtype=torch.bfloat16, device="cuda")
    for i in range(b):
        c["v"][i] = rnd(l, h, p)
    assert c["v"].numel() * 2 > 1 << 32
    y, st = _scan(c, normalize=True, return_states=True)
    assert st.numel() * 4 > 1 << 32
    for i in (0, b - 1):
        one = {k: (v[i:i + 1].contiguous() if k in ("q", "k", "v", "dt", "beta") else v)
               for k, v in c.items()}
        y1, st1 = _scan(one, normalize=True, return_states=True)
        assert torch.equal(y1[0], y[i]) and torch.equal(st1[0], st[i])
    c["dy"], c["d_final"] = y, None
    gr = _bwd(c, st, normalize=True)
    one.update(dy=y[b - 1:].contiguous(), d_final=None)
    g1 = _bwd(one, st1, normalize=True)
    for k in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert torch.equal(gr[k][b - 1], g1[k][0]), k


def test_refusals():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = delta_case(70, 2, 20, 4, 2, 64, 64, "bf16")

    def bad(**over):
        d = dict(c, **over)
        with pytest.raises((ValueError, ssd.SsdError)):
            _scan(d)
    bad(v=c["v"].float())
    bad(v=c["v"].cpu())
    bad(k=c["k"][:, :-1].contiguous())
    bad(q=c["q"].transpose(0, 1))
    bad(beta=c["beta"].float())
    bad(A=c["A"].double())
    bad(dt_bias=c["dt_bias"][:2])
    bad(init=torch.zeros((2, 4, 64, 32), device="cuda"))
    bad(seq=torch.zeros((2, 20), dtype=torch.int64, device="cuda"))
    bad(k=torch.zeros((2, 20, 3, 64), device="cuda", dtype=torch.bfloat16),
        q=torch.zeros((2, 20, 3, 64), device="cuda", dtype=torch.bfloat16))
    bad(v=c["v"][..., :48].contiguous())
    with pytest.raises(ssd.SsdError):
        _scan(c, normalize=True, norm_eps=-1.0)
    with pytest.raises(ssd.SsdError):
        _scan(c, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        _bwd(c, states=torch.zeros((2, 2, 4, 64, 64), device="cuda"))
    with pytest.raises(ValueError):
        ssd.delta_step(torch.zeros((2, 4, 64, 64), device="cuda", dtype=torch.bfloat16),
                       *(c[k] if k == "A" else c[k][:, 0].contiguous() for k in NAMES))
