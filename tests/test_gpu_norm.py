"""The layer norm and its gradient against the fp64 oracle."""
import numpy as np
import pytest

from delta_util import io_dtype, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

# Sums are fp32: dim roundings of 2^-24 in the worst order, far fewer in theirs (a
# lane adds at most 64 or dim / 256 terms, then a tree): 200 * 2^-24 < 1.2e-5.
FINE = 1.2e-5
ONE = 2.0 ** -8 * 1.02  # one rounding to bf16


def _case(seed, rows, dim, io, residual=True):
    torch = torch_mod()
    r = np.random.default_rng(seed)
    dt = io_dtype(io)

    def put(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(dtype)
    lead = rows if isinstance(rows, tuple) else (rows,)
    return dict(x=put(r.normal(size=lead + (dim,)) + 0.5, dt),
                r=put(2 * r.normal(size=lead + (dim,)), dt) if residual else None,
                dy=put(r.normal(size=lead + (dim,)), dt), ds=put(r.normal(size=lead + (dim,)), dt),
                w=put(1 + 0.3 * r.normal(size=dim), torch.float32),
                b=put(0.3 * r.normal(size=dim), torch.float32))


def _np(t):
    return t.double().cpu().numpy()


def check(c, io, what, weight=True, bias=True, eps=1e-5):
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    w, b = (c["w"] if weight else None), (c["b"] if bias else None)
    res = ssd.layer_norm(c["x"], w, b, residual=c["r"], eps=eps, return_stats=True)
    s = c["x"] if c["r"] is None else (c["x"].float() + c["r"].float()).to(c["x"].dtype)
    y, stats = res[0], res[-1]
    if c["r"] is not None:
        assert torch.equal(res[1], s)
    yo, mean, rstd = oracle.layer_norm(_np(s), _np(w) if weight else None,
                                       _np(b) if bias else None, eps)
    got = dict(y=rel(y, yo), rstd=rel(stats[1], rstd.reshape(-1)))
    # a mean is a sum of terms of the row's size, whatever it comes to itself
    got["mean"] = float(np.max(np.abs(_np(stats[0]) - mean.reshape(-1))
                               / np.sqrt((_np(s) ** 2).mean(-1) + 1e-300).reshape(-1), initial=0.0))
    fine = FINE if io == "f32" else ONE
    log(what, got)
    assert got["y"] <= fine and got["rstd"] <= FINE and got["mean"] <= FINE, (what, got)
    g = ssd.layer_norm_bwd(c["dy"], s, stats, w, bias=bias, d_sum=c["ds"])
    o = oracle.layer_norm_grad(_np(c["dy"]), _np(s), _np(w) if weight else None, eps, _np(c["ds"]))
    assert set(g) == {"dx"} | ({"dweight"} if weight else set()) | ({"dbias"} if bias else set())
    for k, x in g.items():
        e = rel(x, o[k])
        log(what, k, "%.2e" % e)
        assert e <= (fine if k == "dx" else FINE), (what, k, e)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [
    (1, 1), (3, 2), (7, 7), (200, 16), (33, 64), (40, 65), (129, 256), (65, 257), (17, 512),
    (1999, 771), (70, 770), (50, 1024), (9, 2048), (300, 2560), (5, 3071), (5, 4096), (11, 4097),
    (6, 8192), (3, 8200), (4, 16384), (3, 16385), (2, 40000), (5000, 48)],
    ids=lambda v: str(v))
def test_norm_and_gradient(rows, dim, io):
    check(_case(rows + dim, rows, dim, io, residual=(rows + dim) % 2 == 0), io, "%dx%d" % (rows, dim))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_without_weight_or_bias_and_more_axes(io):
    c = _case(5, (3, 4, 5), 96, io)
    check(c, io, "axes")
    check(c, io, "no weight", weight=False)
    check(c, io, "no bias", bias=False)
    check(c, io, "neither", weight=False, bias=False)


@pytest.mark.parametrize("dim", [40, 100, 700, 5000, 20000])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_constant_rows_and_far_means(io, dim):
    """Rows of one value give the bias (eps keeps the deviation finite), rows far
    from zero keep their deviation (the squares are taken about the mean)."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    dt = io_dtype(io)
    x = torch.full((3, dim), 0.75, dtype=dt, device="cuda")
    b = torch.arange(dim, device="cuda", dtype=torch.float32)
    y, st = ssd.layer_norm(x, None, b, return_stats=True)
    assert torch.equal(y, b.to(dt).expand(3, dim)) and (st[0] == 0.75).all()
    r = np.random.default_rng(1)
    x = torch.from_numpy((1000 + 8 * r.integers(-3, 4, size=(4, dim))).astype(np.float32)).cuda().to(dt)
    y, st = ssd.layer_norm(x, return_stats=True)
    yo, mean, rstd = oracle.layer_norm(_np(x))
    # the mean's own rounding, 2^-24 * 1000 * a few, moves every element of hat
    assert rel(y, yo) <= (1e-4 if io == "f32" else ONE + 1e-4)
    assert rel(st[1], rstd) <= 1e-4


@pytest.mark.parametrize("dim", [100, 101, 2560, 6000, 20000])
def test_outputs_in_place(dim):
    """The sum over x or the residual, y over the other; dx over dy or d_sum."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for io in ("bf16", "f32"):
        c = _case(dim, 70, dim, io)
        y, s, st = ssd.layer_norm(c["x"], c["w"], c["b"], residual=c["r"], return_stats=True)
        for first in (True, False):
            x, r = c["x"].clone(), c["r"].clone()
            y2, s2 = ssd.layer_norm(x, c["w"], c["b"], residual=r, sum_out=x if first else r,
                                    out=r if first else x)
            assert torch.equal(y2, y) and torch.equal(s2, s)
        x = c["x"].clone()
        assert torch.equal(ssd.layer_norm(x, c["w"], out=x), ssd.layer_norm(c["x"], c["w"]))
        want = ssd.layer_norm_bwd(c["dy"], s, st, c["w"], bias=True, d_sum=c["ds"])
        for name in ("dy", "ds"):
            d = dict(dy=c["dy"].clone(), ds=c["ds"].clone())
            got = ssd.layer_norm_bwd(d["dy"], s, st, c["w"], bias=True, d_sum=d["ds"], out=d[name])
            for k in want:
                assert torch.equal(got[k], want[k]), (io, name, k)


def test_a_row_of_nan_stays_a_row():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for dim in (20, 200, 1000, 5000, 17000):
        x = torch.randn((9, dim), device="cuda")
        want = ssd.layer_norm(x)
        x[4, 3] = float("nan")
        x[6, 5] = float("inf")
        got = ssd.layer_norm(x)
        rows = [0, 1, 2, 3, 5, 7, 8]
        assert torch.equal(got[rows], want[rows]) and torch.isnan(got[[4, 6]]).any(1).all()


def test_unaligned_views_and_guards():
    """Contiguous tensors that start off a 16-byte boundary; nothing beside the
    outputs is written."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    for io in ("bf16", "f32"):
        for dim in (64, 640, 4800, 16400):
            c = _case(dim, 6, dim, io)
            for off in (1, 2, 3):
                def shift(t, fill=None):
                    flat = torch.full((t.numel() + 64,), 3.0, dtype=t.dtype, device="cuda")
                    v = flat[off:off + t.numel()].view(t.shape)
                    if fill is None:
                        v.copy_(t)
                    return flat, v
                fo, o = shift(c["x"], fill=True)
                fs, so = shift(c["x"], fill=True)
                y, s, st = ssd.layer_norm(shift(c["x"])[1], c["w"], c["b"], residual=shift(c["r"])[1],
                                          out=o, sum_out=so, return_stats=True)
                y0, s0, st0 = ssd.layer_norm(c["x"], c["w"], c["b"], residual=c["r"], return_stats=True)
                assert torch.equal(s, s0) and rel(y, _np(y0)) <= 2 * (FINE if io == "f32" else ONE)
                g = ssd.layer_norm_bwd(shift(c["dy"])[1], s, st, c["w"], bias=True, d_sum=shift(c["ds"])[1])
                g0 = ssd.layer_norm_bwd(c["dy"], s0, st0, c["w"], bias=True, d_sum=c["ds"])
                for k in g:
                    assert rel(g[k], _np(g0[k])) <= 2 * (ONE if k == "dx" and io == "bf16" else FINE), k
                for f in (fo, fs):
                    assert (f[:off] == 3.0).all() and (f[off + 6 * dim:] == 3.0).all()


def test_empty_and_refusals():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    x = torch.empty((0, 40), device="cuda")
    y, st = ssd.layer_norm(x, return_stats=True)
    assert y.shape == (0, 40) and st.shape == (2, 0)
    w = torch.ones(40, device="cuda")
    g = ssd.layer_norm_bwd(x, x, st, w, bias=True)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    x = torch.zeros((5, 40), device="cuda")
    for kw in (dict(weight=w[:20]), dict(weight=w.double()), dict(bias=w.cpu()),
               dict(residual=x[:4]), dict(residual=x.bfloat16()), dict(sum_out=x), dict(eps=-1.0)):
        with pytest.raises((ValueError, ssd.SsdError)):
            ssd.layer_norm(x, **kw)
    with pytest.raises(ValueError):
        ssd.layer_norm(x.t())
    with pytest.raises(ValueError):
        ssd.layer_norm(x.half())
    with pytest.raises(ValueError):
        ssd.layer_norm_bwd(x, x, torch.zeros((2, 4), device="cuda"))


def test_graph_and_streams_and_repeats():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = _case(77, 3000, 768, "bf16")

    def work():
        y, s, st = ssd.layer_norm(c["x"], c["w"], c["b"], residual=c["r"], return_stats=True)
        g = ssd.layer_norm_bwd(c["dy"], s, st, c["w"], bias=True, d_sum=c["ds"])
        return [y, s, st, g["dx"], g["dweight"], g["dbias"]]
    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, o in zip(work(), want):
            assert torch.equal(x, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(3):
        new = _case(78 + i, 3000, 768, "bf16")
        for k in c:
            c[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for x, o in zip(got, work()):
            assert torch.equal(x, o)
