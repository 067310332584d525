"""The gated recurrence's chain of tiles in groups of 16 and of 8 tiles (many
sequences of many tiles), forward, gradient and packed, against the fp64 oracle
with the tolerances of test_gpu_gated.py."""
import numpy as np
import pytest

from gpu_util import log, torch_mod
from test_gpu_gated import DELTA, HALF, _case, _close, _np

pytestmark = pytest.mark.gpu


# columns (64 or 128 channels of a sequence) x tiles above 1024: groups of 16
# up to 12 columns, of 8 beyond; odd and even widths
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("docs", [False, True])
@pytest.mark.parametrize("shape", [(6, 26300, 3), (7, 19000, 6), (13, 10200, 5), (20, 6800, 18)],
                         ids=str)
def test_groups_of_tiles(shape, docs, io):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import gated as go
    torch = torch_mod()
    b, l, d = shape
    log("groups of tiles", shape, docs, io)
    c = _case(7000 + b, *shape, io=io)
    if docs:  # documents of about 1500 tokens: some tiles hold none, some one, some two
        rng = np.random.default_rng(7100 + b)
        c["seq"] = torch.from_numpy(np.cumsum(rng.random((b, l)) < 1 / 1500, 1).astype(np.int32)).cuda()
    kw = dict(initial_state=c["init"], seq_idx=c["seq"])
    y, fin, st = ssd.gated_scan(c["x"], c["gates"], c["lam"], return_final_state=True,
                                return_states=True, **kw)
    grads = [ssd.gated_scan_bwd(c["x"], c["gates"], c["lam"], c["dy"], d_final=c["dfin"], states=s,
                                **kw) for s in (None, st)]
    torch.cuda.synchronize()
    n = _np(c)
    r = go.scan(n["x"], n["gates"], n["lam"], 8.0, n["init"], n["seq"], delta=DELTA)
    _close(y, r["y"], r["err"] + HALF[io] * np.abs(r["y"]) * 1.01 + 1e-30, "y")
    _close(fin, r["final"], r["err"][:, -1] + 2.0 ** -24 * np.abs(r["final"]), "final")
    k = go.grad(n["x"], n["gates"], n["lam"], 8.0, n["dy"], n["init"], n["seq"], n["dfin"],
                delta=DELTA)
    for g in grads:
        for key in ("dx", "dgates"):
            _close(g[key], k[key], k["err_" + key] + HALF[io] * np.abs(k[key]) * 1.01 + 1e-30, key)
        _close(g["dlam"], k["dlam"], k["err_dlam"] + 1e-30, "dlam")
        _close(g["d_init"], k["d_init"], k["err_d_init"] + 2.0 ** -23 * np.abs(k["d_init"]) + 1e-30,
               "d_init")
