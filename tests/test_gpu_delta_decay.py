"""The gated delta rule where a state is forgotten inside a chunk: what little reaches
the tokens behind, by itself."""
import numpy as np
import pytest

from delta_util import BOUNDS, as64, delta_case, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "dt", "A", "beta")
CUT = 74  # the token that forgets, the eleventh of the second chunk


def _case(seed, io, n, p, drop, b=2, h=4, g=2, l=190):
    """Token CUT decays the state by e^-drop, every other one by e^-0.02 or less."""
    c = delta_case(seed, b, l, h, g, n, p, io, normalize=True)
    c["dt_bias"] = None
    c["A"] = c["A"] * 0 - 1
    c["dt"] = c["dt"].abs().clamp(max=2.0) * 0.01
    c["dt"][:, CUT] = drop
    return c


def _run(c, grad):
    import mamba_ssd_chunked_chunk_amd as ssd
    args, side = [c[k] for k in NAMES], dict(normalize=True, dt_softplus=False)
    e = as64(c)
    ins = [e[k] for k in NAMES]
    if grad:
        return (ssd.delta_scan_bwd(*args, c["dy"], d_final=c["d_final"], **side),
                oracle.grad(*ins, dy=e["dy"], d_final=e["d_final"], **side))
    y, fin, st = ssd.delta_scan(*args, return_final_state=True, return_states=True, **side)
    return dict(y=y, final=fin, states=st), oracle.scan(*ins, **side)


def _near(x, o, bound, what):
    r = rel(x, o)
    log(*what, "%.2e" % r)
    assert r <= bound, (what, r)


SIZES = [(32, 16, 4), (64, 64, 4), (128, 128, 4), (64, 32, 132)]  # n, p, heads


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("drop", [6.0, 12.0, 16.0, 25.0])
@pytest.mark.parametrize("n,p,h", SIZES)
def test_reads_of_a_forgotten_state(io, drop, n, p, h):
    """Behind the token nothing is written (beta of zero): its chunk's other tokens
    read what is left, and so do the next chunk and the final state."""
    c = _case(3, io, n, p, drop, h=h)
    c["beta"][:, CUT:] = 0
    c["beta"][:, :64] = 0  # and the chunk starts from zero
    got, ref = _run(c, False)
    for part in (slice(CUT, 128), slice(128, None)):
        for hh in range(0, h, 33):
            _near(got["y"][:, part, hh], ref["y"][:, part, hh], BOUNDS[io]["y"], ("y", io, drop, part))
    _near(got["final"], ref["final"], BOUNDS[io]["state"], ("final", io, drop))
    _near(got["states"][:, 1], ref["states"][:, 1], BOUNDS[io]["state"], ("states", io, drop))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,p,h", SIZES)
def test_small_values_behind_large_ones(io, n, p, h):
    """Values of 2^16 in front of a token that decays them to the size of what is
    written behind it: the corrections there are of the inverse's small elements.  (The
    triangle's inverse, two terms off by 2^-22, meets rows 2^16 larger than the result,
    whose own terms are off by 2^-38 of them: as many bits as everywhere.)"""
    c = _case(4, io, n, p, 12.0, h=h)
    c["v"][:, 64:CUT] *= 2.0 ** 16
    got, ref = _run(c, False)
    _near(got["y"][:, CUT:], ref["y"][:, CUT:], BOUNDS[io]["y"], ("y", io))
    _near(got["final"], ref["final"], BOUNDS[io]["state"], ("final", io))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,p,h", SIZES)
def test_gradient_across_a_forgetting_token(io, n, p, h):
    """Cotangents behind the token alone reach the tokens in front of it through the
    small elements of the masked products and of the inverse."""
    c = _case(5, io, n, p, 12.0, h=h)
    c["dy"][:, :CUT] = 0
    c["dy"][:, 128:] = 0
    c["d_final"].zero_()
    got, ref = _run(c, True)
    part = slice(64, CUT)
    for name in ("dv", "dbeta"):
        _near(got[name][:, part], ref[name][:, part], BOUNDS[io][name], (name, io))
