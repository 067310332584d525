"""The gated delta rule's four-wave walk (calls with few columns): what its waves hand
each other through LDS stays apart from one chunk to the next."""
import pytest

from delta_util import BOUNDS, as64, delta_case, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "dt", "A", "beta")


def _scan(c, **kw):
    import mamba_ssd_chunked_chunk_amd as ssd
    return ssd.delta_scan(*(c[k] for k in NAMES), dt_bias=c["dt_bias"], initial_state=c["init"],
                          normalize=True, **kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [32, 64, 128])
def test_long_chains_repeat_and_keep_their_rows(io, n):
    """150 chunks by four waves to 16 columns, with and without the states' stores
    between a chunk's last barrier and its read-out: the same bits each time, and the
    same as from the chunk in the middle on."""
    torch = torch_mod()
    b, l, h, p = 2, 150 * 64 - 7, 4, 32
    c = delta_case(n, b, l, h, 2, n, p, io, normalize=True, init=True)
    y, fin, st = _scan(c, return_final_state=True, return_states=True)
    for _ in range(4):
        y2, fin2 = _scan(c, return_final_state=True)
        assert torch.equal(y, y2) and torch.equal(fin, fin2)
        y2, fin2, st2 = _scan(c, return_final_state=True, return_states=True)
        assert torch.equal(y, y2) and torch.equal(fin, fin2) and torch.equal(st, st2)
    at = 75 * 64
    tail = dict(c, init=st[:, 74].contiguous())
    for k in ("q", "k", "v", "dt", "beta"):
        tail[k] = c[k][:, at:].contiguous()
    y2, fin2 = _scan(tail, return_final_state=True)
    assert torch.equal(y[:, at:], y2) and torch.equal(fin, fin2)
    # the last three chunks against the oracle
    at = 147 * 64
    e = as64(dict(c, init=st[:, 146]))
    for k in ("q", "k", "v", "dt", "beta"):
        e[k] = e[k][:, at:]
    ref = oracle.scan(*(e[k] for k in NAMES), dt_bias=e["dt_bias"], init=e["init"], normalize=True)
    r = rel(y[:, at:], ref["y"]), rel(fin, ref["final"])
    log("long chain", io, n, *("%.2e" % x for x in r))
    assert r[0] <= BOUNDS[io]["y"] and r[1] <= BOUNDS[io]["state"]
