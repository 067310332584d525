"""Argument checks of ssd_linear, ssd_linear_bwd and the gated recurrence that
need no GPU: every refused call returns its status before the HIP runtime is
touched."""
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from mamba_ssd_chunked_chunk_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def lib(L):
    try:
        return L.load()
    except L.LibraryMissing:
        from mamba_ssd_chunked_chunk_amd import build
        build.build(verbose=False)
        return L.load()


def test_constants_match_the_header(L):
    text = open(os.path.join(ROOT, "include", "ssd.h")).read()
    assert int(re.search(r"#define SSD_GATED_CHUNK (\d+)", text).group(1)) == L.SSD_GATED_CHUNK
    for name, code in L.ACTIVATIONS.items():
        assert re.search(r"SSD_ACT_%s = %d\b" % (name.upper(), code), text), name


def test_linear_refusals(lib, L):
    def lin(**over):
        kw = dict(x=FAKE, w=FAKE, b=None, r=None, o=FAKE, p=None, act=0, m=300, k=64, n=40, io=1,
                  ws=FAKE, wsb=1 << 40)
        kw.update(over)
        return lib.ssd_linear(kw["x"], kw["w"], kw["b"], kw["r"], kw["o"], kw["p"], kw["act"],
                              kw["m"], kw["k"], kw["n"], kw["io"], kw["ws"], kw["wsb"], None)
    assert lin(io=2) == L.SSD_ERR_UNSUPPORTED
    assert lin(act=4) == L.SSD_ERR_UNSUPPORTED
    assert lin(act=-1) == L.SSD_ERR_UNSUPPORTED
    assert lin(m=-1) == L.SSD_ERR_SHAPE
    assert lin(k=0) == L.SSD_ERR_SHAPE
    assert lin(n=-4) == L.SSD_ERR_SHAPE
    assert lin(k=(1 << 20) + 1) == L.SSD_ERR_UNSUPPORTED
    assert lin(m=1 << 31) == L.SSD_ERR_UNSUPPORTED
    assert lin(m=1 << 30, k=1, n=1) == L.SSD_ERR_UNSUPPORTED    # rows of one element, padded
    for name in ("x", "w", "o"):
        assert lin(**{name: None}) == L.SSD_ERR_NULL
    # each tensor as its rows are among themselves: 64 and 40 bf16 values are
    # multiples of 16 bytes, 36 of 8, odd widths of 2
    for name in ("x", "w", "o", "r", "p"):
        assert lin(**{name: FAKE + 8}) == L.SSD_ERR_ALIGN
    for name in ("o", "r", "p"):
        assert lin(n=36, **{name: FAKE + 4}) == L.SSD_ERR_ALIGN
        assert lin(n=37, **{name: FAKE + 1}) == L.SSD_ERR_ALIGN
    assert lin(k=37, x=FAKE + 1) == L.SSD_ERR_ALIGN
    assert lin(b=FAKE + 2) == L.SSD_ERR_ALIGN
    # odd widths are laid out again in the workspace
    need = lib.ssd_linear_workspace_bytes(300, 65, 40, 1)
    assert need >= (300 + 40) * 72 * 2
    assert lin(k=65, wsb=need - 1) == L.SSD_ERR_WORKSPACE
    assert lin(k=65, ws=None) == L.SSD_ERR_WORKSPACE
    assert lin(k=65, ws=FAKE + 16) == L.SSD_ERR_ALIGN
    assert lin(m=0, x=None) == L.SSD_OK
    ws = lib.ssd_linear_workspace_bytes
    assert ws(0, 64, 64, 1) == 0 and ws(40, 0, 64, 1) == 0 and ws(40, 65, 64, 5) == 0
    assert ws(40, 65, 64, 1) == ws(40, 65, 64, 1) > 0


def test_linear_bwd_refusals(lib, L):
    def bwd(**over):
        kw = dict(dy=FAKE, x=FAKE, w=FAKE, pre=FAKE, act=2, dx=FAKE, dw=FAKE, db=FAKE, m=300,
                  k=64, n=40, io=1, ws=FAKE, wsb=1 << 40)
        kw.update(over)
        return lib.ssd_linear_bwd(kw["dy"], kw["x"], kw["w"], kw["pre"], kw["act"], kw["dx"],
                                  kw["dw"], kw["db"], kw["m"], kw["k"], kw["n"], kw["io"],
                                  kw["ws"], kw["wsb"], None)
    assert bwd(io=9) == L.SSD_ERR_UNSUPPORTED
    assert bwd(act=7) == L.SSD_ERR_UNSUPPORTED
    assert bwd(m=-1) == L.SSD_ERR_SHAPE
    assert bwd(n=0) == L.SSD_ERR_SHAPE
    assert bwd(pre=None) == L.SSD_ERR_NULL
    assert bwd(dy=None) == L.SSD_ERR_NULL
    assert bwd(x=None) == L.SSD_ERR_NULL
    assert bwd(w=None) == L.SSD_ERR_NULL
    for name in ("dy", "x", "w", "pre", "dx", "dw"):
        assert bwd(**{name: FAKE + 4}) == L.SSD_ERR_ALIGN
    assert bwd(db=FAKE + 2) == L.SSD_ERR_ALIGN
    need = lib.ssd_linear_bwd_workspace_bytes(300, 64, 40, 2, 1)
    assert need >= 300 * 40 * 2
    assert bwd(wsb=need - 1) == L.SSD_ERR_WORKSPACE
    assert bwd(ws=None) == L.SSD_ERR_WORKSPACE
    assert lib.ssd_linear_bwd_workspace_bytes(300, 64, 40, 9, 1) == 0


def test_gated_refusals(lib, L):
    def scan(**over):
        kw = dict(x=FAKE, g=FAKE, lam=FAKE, scale=8.0, init=None, seq=None, y=FAKE, fin=None,
                  st=None, b=2, l=200, d=36, io=1, ws=FAKE, wsb=1 << 40)
        kw.update(over)
        return lib.ssd_gated_scan(kw["x"], kw["g"], kw["lam"], kw["scale"], kw["init"], kw["seq"],
                                  kw["y"], kw["fin"], kw["st"], kw["b"], kw["l"], kw["d"],
                                  kw["io"], kw["ws"], kw["wsb"], None)

    def bwd(**over):
        kw = dict(x=FAKE, g=FAKE, lam=FAKE, scale=8.0, init=None, seq=None, st=None, dy=FAKE,
                  df=None, dx=FAKE, dg=FAKE, dl=FAKE, di=None, b=2, l=200, d=36, io=1, ws=FAKE,
                  wsb=1 << 40)
        kw.update(over)
        return lib.ssd_gated_scan_bwd(kw["x"], kw["g"], kw["lam"], kw["scale"], kw["init"],
                                      kw["seq"], kw["st"], kw["dy"], kw["df"], kw["dx"], kw["dg"],
                                      kw["dl"], kw["di"], kw["b"], kw["l"], kw["d"], kw["io"],
                                      kw["ws"], kw["wsb"], None)
    for f in (scan, bwd):
        assert f(io=3) == L.SSD_ERR_UNSUPPORTED
        assert f(b=-1) == L.SSD_ERR_SHAPE
        assert f(l=-1) == L.SSD_ERR_SHAPE
        assert f(d=0) == L.SSD_ERR_SHAPE
        assert f(scale=-1.0) == L.SSD_ERR_SHAPE
        assert f(scale=math.inf) == L.SSD_ERR_SHAPE
        assert f(scale=math.nan) == L.SSD_ERR_SHAPE
        assert f(b=70000) == L.SSD_ERR_UNSUPPORTED
        assert f(b=64, l=1 << 20, d=1 << 16) == L.SSD_ERR_UNSUPPORTED   # 2^42 elements
        assert f(x=None) == L.SSD_ERR_NULL
        assert f(g=None) == L.SSD_ERR_NULL
        assert f(lam=None) == L.SSD_ERR_NULL
        for name in ("x", "g"):
            assert f(**{name: FAKE + 1}) == L.SSD_ERR_ALIGN
            assert f(io=0, **{name: FAKE + 2}) == L.SSD_ERR_ALIGN
        for name in ("lam", "init", "st"):
            assert f(**{name: FAKE + 2}) == L.SSD_ERR_ALIGN
        assert f(seq=FAKE + 2) == L.SSD_ERR_ALIGN
        assert f(ws=FAKE + 64) == L.SSD_ERR_ALIGN
        assert f(ws=None) == L.SSD_ERR_WORKSPACE
        assert f(wsb=100) == L.SSD_ERR_WORKSPACE
    assert scan(y=None) == L.SSD_ERR_NULL
    assert scan(b=0, x=None) == L.SSD_OK
    assert scan(l=0, x=None) == L.SSD_OK
    assert bwd(dy=None) == L.SSD_ERR_NULL
    assert bwd(dl=None) == L.SSD_ERR_NULL
    assert bwd(l=0) == L.SSD_ERR_SHAPE
    assert bwd(dx=FAKE + 1) == L.SSD_ERR_ALIGN
    q = lib.ssd_gated_scan_workspace_bytes
    assert q(2, 200, 36) > 0 and q(0, 5, 5) == 0 and q(2, 0, 5) == 0
    assert lib.ssd_gated_scan_bwd_workspace_bytes(2, 200, 36) >= q(2, 200, 36)

    def step(**over):
        kw = dict(s=FAKE, x=FAKE, g=FAKE, lam=FAKE, scale=8.0, y=FAKE, b=2, d=36, io=1)
        kw.update(over)
        return lib.ssd_gated_step(kw["s"], kw["x"], kw["g"], kw["lam"], kw["scale"], kw["y"],
                                  kw["b"], kw["d"], kw["io"], None)
    assert step(io=-1) == L.SSD_ERR_UNSUPPORTED
    assert step(b=-1) == L.SSD_ERR_SHAPE
    assert step(d=0) == L.SSD_ERR_SHAPE
    assert step(scale=math.nan) == L.SSD_ERR_SHAPE
    for name in ("s", "x", "g", "lam", "y"):
        assert step(**{name: None}) == L.SSD_ERR_NULL
        assert step(**{name: FAKE + 1}) == L.SSD_ERR_ALIGN
    assert step(b=1 << 20, d=1 << 14) == L.SSD_ERR_UNSUPPORTED
    assert step(b=0) == L.SSD_OK


def test_binding_refusals_on_the_host():
    """The binding's own checks, on CPU tensors: no GPU is asked for anything."""
    import torch

    import mamba_ssd_chunked_chunk_amd as ssd
    x, w = torch.zeros(4, 8), torch.zeros(3, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssd.linear(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssd.linear_bwd(x, x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssd.gated_scan(torch.zeros(1, 2, 3), torch.zeros(1, 2, 6), torch.zeros(3))
    with pytest.raises(ValueError, match="seqlen"):
        ssd.gated_scan_bwd(x, x, x, x)
    with pytest.raises(ValueError, match="dim"):
        ssd.gated_step(torch.zeros(1, 3), torch.zeros(3), torch.zeros(6), torch.zeros(3))
