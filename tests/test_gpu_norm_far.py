"""The layer norm of rows far from zero: what little they deviate by is not lost in the
rounding of their mean."""
import numpy as np
import pytest

from gpu_util import log, torch_mod
from oracle import delta as oracle

pytestmark = pytest.mark.gpu

DIMS = [5, 40, 100, 771, 2560, 5000, 10000, 20000]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dim", DIMS)
def test_rows_of_one_value_give_the_bias(io, dim):
    """Whatever the value: s - mean is some roundings of it at first, the mean of which
    is then taken off too, so that 2^-22 of them is left (dim roundings of 2^-24 each
    at most in the worst order, far fewer in this one: 16 of 2^-24 of the value first,
    and of that again)."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    value = [1000.1, -1234.567, 3.3, 40000.7, 1e-3]
    x = torch.tensor(value, device="cuda").to(torch.float32 if io == "f32" else torch.bfloat16)
    x = x[:, None].expand(len(value), dim).contiguous()
    y, st = ssd.layer_norm(x, return_stats=True)
    size = np.abs(x[:, 0].double().cpu().numpy())
    off = np.abs(y.double().cpu().numpy()).max(1)
    log("one value", io, dim, off)
    # 1 / deviation is 1 / sqrt(eps) = 317
    assert (off <= 317 * (16 * 2.0 ** -24) ** 2 * size + 1e-12).all(), off
    np.testing.assert_allclose(st[0].double().cpu().numpy(), x[:, 0].double().cpu().numpy(),
                               rtol=2.0 ** -23)
    np.testing.assert_allclose(st[1].double().cpu().numpy(), 1e5 ** 0.5, rtol=1e-6)


@pytest.mark.parametrize("dim", DIMS)
def test_small_deviations_far_from_zero(dim):
    """Rows at 10^4 that deviate by one, in steps that fp32 has there: the differences
    from the rounded mean are exact, and all sums behind them are of their size (100
    roundings of 2^-24 of the deviation in their longest chain: 1e-5)."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    r = np.random.default_rng(dim)
    x = (1e4 + np.round(r.normal(size=(7, dim)) * 512) / 512).astype(np.float32)
    y, st = ssd.layer_norm(torch.from_numpy(x).cuda(), return_stats=True)
    yo, mean, rstd = oracle.layer_norm(x)
    off = np.linalg.norm(y.double().cpu().numpy() - yo) / np.linalg.norm(yo)
    log("far", dim, "%.2e" % off)
    assert off <= 1e-5
    np.testing.assert_allclose(st[1].double().cpu().numpy(), rstd, rtol=1e-5)
    np.testing.assert_allclose(st[0].double().cpu().numpy(), mean, rtol=2.0 ** -23)
