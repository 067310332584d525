"""With bf16 io the gated delta rule's outputs are the fp64 oracle's, rounded once."""
import pytest

from delta_util import FINE, as64, delta_case, rel
from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "dt", "A", "beta")

# Values off by FINE of their size in front of the rounding, whose steps are at least
# 2^-8 of it, reach the next step in one of 2^-8 / FINE cases and are then off by a step
# (2^-7 at most): 2^-7 sqrt(2^8 FINE) of the norm.  An operand of one fp16 term (2^-12 of
# a value on average) in place of two would leave 2^-7 sqrt(2^-4), 4 times as much.
LIMIT = 2.0 ** -7 * (2.0 ** 8 * FINE) ** 0.5


@pytest.mark.parametrize("shape", [(2, 300, 4, 2, 128, 128), (1, 200, 6, 2, 64, 32), (2, 130, 132, 4, 32, 16),
                                   (1, 190, 80, 80, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_outputs_are_rounded_once(shape):
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    c = delta_case(sum(shape) + 1, *shape, "bf16", normalize=True, init=True)
    args, e = [c[k] for k in NAMES], as64(c)
    y = ssd.delta_scan(*args, dt_bias=c["dt_bias"], normalize=True, initial_state=c["init"])
    got = ssd.delta_scan_bwd(*args, c["dy"], dt_bias=c["dt_bias"], normalize=True,
                             initial_state=c["init"], d_final=c["d_final"])
    inputs = dict(dt_bias=e["dt_bias"], normalize=True, init=e["init"])
    ref = oracle.grad(*(e[k] for k in NAMES), dy=e["dy"], d_final=e["d_final"], **inputs)
    ref["y"] = oracle.scan(*(e[k] for k in NAMES), **inputs)["y"]
    for name, x in dict(got, y=y).items():
        if x.dtype != torch.bfloat16:
            continue
        o = torch.from_numpy(ref[name]).bfloat16().double().numpy()
        r = rel(x, o)
        log("rounded once", name, shape, "%.2e" % r)
        assert r <= LIMIT, (name, r)
