"""The gated delta rule where what a chunk starts from is large and its tokens overwrite
it: the state's part of an output and the tokens' part nearly cancel."""
import numpy as np
import pytest
from scipy.linalg import hadamard

from delta_util import FINE, as64, delta_case, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "dt", "A", "beta")
SIZE = 256.0  # of the state in front, beside values of one


def _case(seed, io, p, h, l=64):
    """32 orthogonal keys, each written at full strength: from token 32 on nothing is
    left of the state in front."""
    torch = torch_mod()
    c = delta_case(seed, 2, l, h, 2, 32, p, io, normalize=True, init=True)
    order = np.random.default_rng(seed).permutation(32)
    rows = hadamard(32)[order][np.arange(l) % 32].astype(np.float32)
    c["k"] = torch.from_numpy(rows)[None, :, None].expand_as(c["k"]).to(c["k"])
    c["beta"] = torch.ones_like(c["beta"])
    c["A"] = c["A"] * 0.01
    c["init"] = c["init"] / 0.3 * SIZE
    return c


# The two parts are SIZE times their sum; both are made of two-term operands (FINE of
# the parts), and bf16 outputs are rounded once more.
LIMIT = {"f32": SIZE * FINE, "bf16": SIZE * FINE + 2.0 ** -8}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("p,h", [(16, 4), (64, 4), (32, 264), (128, 40)])
def test_outputs_of_an_overwritten_state(io, p, h):
    import mamba_ssd_chunked_chunk_amd as ssd
    c = _case(p + h, io, p, h)
    y, fin = ssd.delta_scan(*(c[k] for k in NAMES), dt_bias=c["dt_bias"], normalize=True,
                            initial_state=c["init"], return_final_state=True)
    e = as64(c)
    ref = oracle.scan(*(e[k] for k in NAMES), dt_bias=e["dt_bias"], normalize=True, init=e["init"])
    assert np.abs(ref["final"]).max() < 16
    for what, x, o, bound in (("y", y[:, 32:], ref["y"][:, 32:], LIMIT[io]),
                              ("final", fin, ref["final"], LIMIT["f32"])):
        r = rel(x, o)
        log("overwritten", what, io, p, h, "%.2e" % r)
        assert r <= bound, (what, r)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("p,h", [(16, 4), (64, 4), (32, 264), (128, 40)])
def test_gradients_of_an_overwritten_state(io, p, h):
    import mamba_ssd_chunked_chunk_amd as ssd
    c = _case(p + h + 1, io, p, h)
    args, e = [c[k] for k in NAMES], as64(c)
    got = ssd.delta_scan_bwd(*args, c["dy"], dt_bias=c["dt_bias"], normalize=True,
                             initial_state=c["init"], d_final=c["d_final"])
    ref = oracle.grad(*(e[k] for k in NAMES), dy=e["dy"], dt_bias=e["dt_bias"], normalize=True,
                      init=e["init"], d_final=e["d_final"])
    for name in ("dq", "dk", "dbeta"):
        r = rel(got[name][:, 32:], ref[name][:, 32:])
        log("overwritten", name, io, p, h, "%.2e" % r)
        # dk has two such sums over the chunk's tokens, of u and of the state's read
        assert r <= (2 if name == "dk" else 1) * LIMIT[io], (name, r)
