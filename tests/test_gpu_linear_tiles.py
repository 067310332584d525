"""The linear layer's larger tiles, its few rows on both sides of the choice,
and the tails of GELU, against fp64.

The sizes are ones for which the choice of tile and parts takes, bf16 and fp32:
128 x 192 and 128 x 128 forward, and in the gradient both with and without
contraction parts of either product, with whole tiles, ragged ones and widths
off every vector.  Tolerances as in test_gpu_linear.py.
"""
import numpy as np
import pytest

from gpu_util import log, to_f64, torch_mod
from test_gpu_linear import HALF, _close, _linear, _rand

pytestmark = pytest.mark.gpu


# 128 x 128: the first four; 128 x 192: the others (bf16); fp32 takes 128 x 128
# for the sizes with 5000 and more columns
FORWARD = [(6007, 520, 1000), (6016, 192, 1024), (1501, 300, 5003), (1500, 72, 5000),
           (2050, 72, 2000), (2051, 1000, 2001), (3000, 640, 3000), (5999, 200, 1031)]


@pytest.mark.parametrize("act,pre", [("none", False), ("gelu", True)])
@pytest.mark.parametrize("shape", FORWARD, ids=str)
def test_large_tiles(shape, act, pre):
    _linear(*shape, io="bf16", act=act, bias=pre, residual=True, pre=pre,
            seed=3000 + 10 * FORWARD.index(shape))


@pytest.mark.parametrize("shape", [(1501, 300, 5003), (1500, 72, 5000)], ids=str)
def test_large_tiles_fp32(shape):
    _linear(*shape, io="f32", act="silu", bias=True, residual=True, pre=True, seed=3200)


# more than four rows of x against a large weight of odd rows: laid out again first
@pytest.mark.parametrize("shape", [(5, 2561, 1000), (16, 2561, 1031), (17, 1031, 2311),
                                   (32, 4097, 777)], ids=str)
def test_few_rows_laid_out_again(shape):
    _linear(*shape, io="bf16", act="silu", pre=True, seed=3300)


# (rows, in, out): the tile of bf16 and of fp32, and the parts of dx and dW
BACKWARD = [(1030, 2050, 1000),   # 192 without parts
            (1500, 2050, 500),    # 192, dW in 2; 128, dW in 3
            (1500, 2050, 200),    # 192, dW in 4; 128, dW in 8
            (300, 2050, 1552),    # 192, dx in 3
            (4100, 777, 500),     # 128, dW in 8
            (700, 777, 4097),     # 128, dx in 6
            (2500, 260, 5000),    # 128, dx in 4 and dW in 2
            (1500, 2050, 1552)]   # 128 without parts


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", BACKWARD, ids=str)
def test_large_tiles_gradient(shape, io):
    import mamba_ssd_chunked_chunk_amd as ssd
    from oracle import linear as lo
    torch = torch_mod()
    m, k, n = shape
    j = BACKWARD.index(shape)
    act = ["silu", "none", "gelu"][j % 3]
    x, w = _rand(3400 + j, io, m, k), _rand(3500 + j, io, n, k, std=n ** -0.5)
    dy, pre = _rand(3600 + j, io, m, n), _rand(3700 + j, io, m, n, std=2.0)
    log("linear_bwd", m, k, n, io, act)
    g = ssd.linear_bwd(dy, x, w, pre=None if act == "none" else pre, activation=act, bias=True)
    torch.cuda.synchronize()
    xo, wo, eo, po = to_f64(x), to_f64(w), to_f64(dy), to_f64(pre)
    r = lo.linear_grad(eo, xo, wo, po, act)
    ea = np.abs(r["e"])
    ev = np.zeros_like(ea) if act == "none" else 2.0 ** -20 * np.abs(eo) * (1 + np.abs(po))
    er = ev + (HALF[io] if act != "none" else 0) * ea
    for key, by_e, mag, terms in (
            ("dx", er @ np.abs(wo), ea @ np.abs(wo), n),
            ("dweight", er.T @ np.abs(xo), ea.T @ np.abs(xo), m)):
        o = r[key]
        _close(g[key], o, 1.01 * (by_e + (terms + 4) * 2.0 ** -24 * mag + HALF[io] * np.abs(o)), key)
    _close(g["dbias"], r["dbias"],
           (ev.sum(0) + (m + 4) * 2.0 ** -24 * ea.sum(0)) * 1.01 + 1e-30, "dbias")


def test_gelu_tail():
    """GELU and its gradient in fp32 from -3 to -8, relative to their terms.
    Phi's polynomial is off by at most 1.12e-5 of Phi there; the exponential's
    argument, up to 46 binary orders, is rounded three times: 46 ln 2 x 2.5 x
    2^-24 = 4.8e-6; everything else a few 2^-24.  Below 2^-15 = 3.05e-5."""
    import mamba_ssd_chunked_chunk_amd as ssd
    from scipy.special import ndtr
    torch = torch_mod()
    v = np.linspace(-8, -3, 20001).astype(np.float32)
    x = torch.zeros((v.size, 4), device="cuda")
    x[:, 0] = torch.from_numpy(v).cuda()
    w = torch.zeros((4, 4), device="cuda")
    w[:, 0] = 1
    y, pre = ssd.linear(x, w, activation="gelu", return_pre=True)
    dy = torch.zeros_like(y)
    dy[:, 0] = 1
    g = ssd.linear_bwd(dy, x, w, pre=pre, activation="gelu")
    torch.cuda.synchronize()
    z = v.astype(np.float64)
    phi, dens = ndtr(z), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    assert np.array_equal(to_f64(pre)[:, 0], z)
    _close(y[:, 0], z * phi, 2.0 ** -15 * np.abs(z * phi), "gelu")
    _close(g["dx"][:, 0], phi + z * dens, 2.0 ** -15 * (phi + np.abs(z) * dens), "its gradient")


# few rows by the tiles: long contractions and large weights, rows of odd width
# among them, and one size on each side of the choice; bf16, then fp32 sizes
@pytest.mark.parametrize("shape,io", [
    ((1, 16384, 256), "bf16"), ((3, 16385, 250), "bf16"), ((16, 8192, 520), "bf16"),
    ((17, 2560, 4900), "bf16"), ((17, 2560, 4800), "bf16"), ((32, 2561, 10576), "bf16"),
    ((31, 768, 16400), "bf16"), ((2, 20000, 1), "bf16"),
    ((1, 4100, 2048), "f32"), ((1, 4096, 2048), "f32"), ((5, 16384, 130), "f32"),
    ((17, 4096, 36), "f32"), ((20, 4092, 4100), "f32"), ((24, 2560, 7001), "f32"),
    ((19, 4101, 300), "f32")], ids=str)
def test_few_rows_by_the_tiles(shape, io):
    _linear(*shape, io=io, act="gelu", bias=True, residual=True, pre=True, seed=3800)
