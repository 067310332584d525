"""The gated delta rule where rows of q and k are zeros or nearly so: the outputs of
these rows alone, which next to the others' would not show."""
import numpy as np
import pytest

from delta_util import BOUNDS, as64, delta_case, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "dt", "A", "beta")


def _rows(seed, n, p, io, size, h=4, g=2):
    """Every fourth row of q and every fifth of k `size` times as large."""
    c = delta_case(seed, 2, 150, h, g, n, p, io, normalize=True, init=True, packed=True)
    for name, step in (("q", 4), ("k", 5)):
        c[name] = c[name].clone()
        c[name][:, ::step] *= size
    return c


def _check(c, io, what, step=True, **kw):
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    args = [c[k] for k in NAMES]
    side = dict(dt_bias=c["dt_bias"], normalize=True, **kw)
    y, fin, st = ssd.delta_scan(*args, initial_state=c["init"], seq_idx=c["seq"],
                                return_final_state=True, return_states=True, **side)
    got = ssd.delta_scan_bwd(*args, c["dy"], initial_state=c["init"], seq_idx=c["seq"],
                             d_final=c["d_final"], states=st, **side)
    e = as64(c)
    inputs = dict(init=e["init"], seq=e["seq"], **dict(side, dt_bias=e["dt_bias"]))
    ref = oracle.scan(*(e[k] for k in NAMES), **inputs)
    rg = oracle.grad(*(e[k] for k in NAMES), dy=e["dy"], d_final=e["d_final"], **inputs)
    few = dict(dq=slice(None, None, 4), dk=slice(None, None, 5))
    rest = {k: [t for t in range(150) if t % s.step] for k, s in few.items()}
    for name, o in rg.items():
        for part in ((few[name], rest[name]) if name in few else (slice(None),)):
            r = rel(got[name][:, part] if name in few else got[name],
                    o[:, part] if name in few else o)
            log(what, name, "%.2e" % r)
            assert r <= BOUNDS[io][name], (what, name, r)
    for part in (few["dq"], rest["dq"]):
        r = rel(y[:, part], ref["y"][:, part])
        assert r <= BOUNDS[io]["y"], (what, "y", r)
    assert rel(fin, ref["final"]) <= BOUNDS[io]["state"]
    assert rel(st, ref["states"]) <= BOUNDS[io]["state"]
    # one token in the manner of a decode step: those of q, of k, and of both
    for t in (4, 5, 20):
        state = torch.from_numpy(np.ascontiguousarray(ref["states"][:, 1], np.float32)).cuda()
        before = state.double().cpu().numpy()
        tok = [c[k] if k == "A" else c[k][:, t].contiguous() for k in NAMES]
        ys = ssd.delta_step(state, *tok, **side)
        yo, so = oracle.step(before, *(e[k] if k == "A" else e[k][:, t] for k in NAMES),
                             **dict(side, dt_bias=e["dt_bias"]))
        # (y of a small q with a small state is below fp32's normal range: there each of
        # the n products and sums is off by up to 2^-150 of its own, whatever its size, and
        # its rounding to bf16, whose values there are 2^-133 apart, by 2^-134)
        lost = c["k"].shape[-1] * 2.0 ** -150 + (2.0 ** -134 if io == "bf16" else 0)
        off = np.maximum(np.abs(ys.double().cpu().numpy() - yo) - lost, 0)
        assert rel(state, so) < 1e-6, t
        assert np.linalg.norm(off) <= (2e-6 if io == "f32" else 2.0 ** -8) * np.linalg.norm(yo), t


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,p", [(32, 16), (64, 64), (128, 128)])
def test_rows_of_zeros(io, n, p):
    """x / sqrt(|x|^2 + eps) has the derivative 1 / sqrt(eps) at zero."""
    _check(_rows(n, n, p, io, 0.0), io, "zeros %d %d" % (n, p))
    # more columns than one walk's four waves to sixteen of them take
    _check(_rows(n + 1, n, p, io, 0.0, h=132, g=4), io, "zeros %d %d, many heads" % (n, p))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size,eps", [(1e-25, 1e-6), (1e-36, 1e-6), (1e-12, 1e-6), (1e-18, 1e-36),
                                      (1e-18, 1e25)])
def test_small_rows(io, size, eps):
    """Rows that eps outweighs by far, by a little or not at all, down to where their
    squares and eps in units of them leave fp32's range."""
    _check(_rows(5, 64, 32, io, size), io, "size %g eps %g" % (size, eps), norm_eps=eps)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-25, 1e25])
def test_rows_of_every_size_without_eps(io, size):
    """Divided by their norm, rows of any size are alike, their products among
    themselves (1e-50, 1e50) too."""
    c = _rows(6, 64, 32, io, size)
    _check(c, io, "size %g without eps" % size, norm_eps=0.0)
    for k in ("q", "k"):
        c[k] = c[k] * (1 / size if size > 1 else size ** 0.5)
    _check(c, io, "sizes to %g without eps" % size, norm_eps=0.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("l", [200, 65, 64 + 63])
def test_small_keys_in_a_chunk_that_ends_early(io, l):
    """Keys of 1e-8 that are not normalised (beta 1e16 times as large), in a last chunk
    of few tokens: the rows that are not there do not count as keys of one, nor do
    rows of zeros among the others."""
    import mamba_ssd_chunked_chunk_amd as ssd
    for h, g in ((4, 2), (136, 4)):
        c = delta_case(l, 2, l, h, g, 64, 32, io, init=True)
        c["k"], c["beta"], c["init"] = c["k"] * 1e-8, c["beta"] * 1e16, c["init"] * 1e8
        c["k"][:, l - 1] = 0
        args, e = [c[k] for k in NAMES], as64(c)
        y, fin = ssd.delta_scan(*args, dt_bias=c["dt_bias"], initial_state=c["init"],
                                return_final_state=True)
        ref = oracle.scan(*(e[k] for k in NAMES), dt_bias=e["dt_bias"], init=e["init"])
        for t in range(l - l % 64, l):
            r = rel(y[:, t], ref["y"][:, t])
            assert r <= BOUNDS[io]["y"], (h, t, r)
        r = rel(fin, ref["final"])
        log("small keys", io, l, h, "%.2e" % r)
        assert r <= BOUNDS[io]["state"], (h, r)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-10, 1.0, 1e12])
def test_gradient_of_keys_of_every_size(io, size):
    """Keys that are not normalised, some of them zeros, with a beta of the inverse
    square of their size: beta's square (1e40, 1e-48) need not be in fp32's range."""
    import mamba_ssd_chunked_chunk_amd as ssd
    for h, g in ((4, 2), (136, 4)):
        c = delta_case(9, 1, 150, h, g, 64, 32, io, init=True)
        c["k"], c["beta"] = c["k"] * size, c["beta"] / size / size
        c["init"] = c["init"] / size
        c["k"][:, 3::7] = 0
        args, e = [c[k] for k in NAMES], as64(c)
        got = ssd.delta_scan_bwd(*args, c["dy"], dt_bias=c["dt_bias"], initial_state=c["init"])
        ref = oracle.grad(*(e[k] for k in NAMES), dy=e["dy"], dt_bias=e["dt_bias"], init=e["init"])
        for name, o in ref.items():
            r = rel(got[name], o)
            log("keys of", size, name, io, h, "%.2e" % r)
            assert r <= BOUNDS[io][name], (name, h, r)
