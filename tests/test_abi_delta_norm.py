"""Argument checks of the gated delta rule and the layer norm that need no GPU:
every refused call returns its status before the HIP runtime is touched."""
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
    assert int(re.search(r"#define SSD_DELTA_CHUNK (\d+)", text).group(1)) == L.SSD_DELTA_CHUNK


RULE = dict(q=FAKE, k=FAKE, v=FAKE, dt=FAKE, A=FAKE, bias=FAKE, sp=1, lo=0.0, hi=math.inf,
            beta=FAKE, scale=0.1, norm=1, eps=1e-6)
SIZE = dict(b=2, l=100, h=4, p=64, n=128, g=2, io=1)
END = dict(ws=FAKE, wsb=1 << 40)


def _shared(call, L, empty):
    """Refusals that the scan, its gradient and the step share."""
    assert call(io=2) == L.SSD_ERR_UNSUPPORTED
    for bad in (dict(b=-1), dict(h=0), dict(g=0), dict(h=4, g=3), dict(p=0), dict(n=-32),
                dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan)):
        assert call(**bad) == L.SSD_ERR_SHAPE, bad
    assert call(eps=math.nan, norm=0, v=None) == L.SSD_ERR_NULL  # not used then
    for bad in (dict(p=48), dict(p=256), dict(n=16), dict(n=96), dict(n=256), dict(h=1 << 15, g=1)):
        assert call(**bad) == L.SSD_ERR_UNSUPPORTED, bad
    for name in ("q", "k", "v", "dt", "A", "beta"):
        assert call(**{name: None}) == L.SSD_ERR_NULL, name
    assert call(A=FAKE + 2) == L.SSD_ERR_ALIGN
    assert call(bias=FAKE + 2) == L.SSD_ERR_ALIGN
    assert call(dt=FAKE + 1) == L.SSD_ERR_ALIGN
    assert call(beta=FAKE + 2, io=0) == L.SSD_ERR_ALIGN
    assert call(**empty) == L.SSD_OK


def test_delta_scan_refusals(lib, L):
    def call(**over):
        kw = {**RULE, **SIZE, **END, **dict(init=None, seq=None, y=FAKE, fin=FAKE, st=None), **over}
        return lib.ssd_delta_scan(*(kw[k] for k in (*RULE, "init", "seq", "y", "fin", "st",
                                                    *SIZE, *END)), None)
    _shared(call, L, dict(b=0, v=None))
    assert call(l=-1) == L.SSD_ERR_SHAPE
    assert call(y=None) == L.SSD_ERR_NULL
    assert call(b=70000) == L.SSD_ERR_UNSUPPORTED
    assert call(l=(1 << 28) + 1) == L.SSD_ERR_UNSUPPORTED
    assert call(b=2, h=4, l=1 << 27) == L.SSD_ERR_UNSUPPORTED  # chunks and heads
    for name in ("q", "k", "v", "y", "init", "fin", "st"):
        assert call(**{name: FAKE + 8}) == L.SSD_ERR_ALIGN, name
    assert call(seq=FAKE + 2) == L.SSD_ERR_ALIGN
    need = lib.ssd_delta_scan_workspace_bytes(2, 100, 4, 64, 128, 2, 1)
    assert need > 0
    assert call(wsb=need - 1) == L.SSD_ERR_WORKSPACE
    assert call(ws=None) == L.SSD_ERR_WORKSPACE
    assert call(ws=FAKE + 128) == L.SSD_ERR_ALIGN
    assert call(l=0, fin=None, v=None, ws=None) == L.SSD_OK
    ws = lib.ssd_delta_scan_workspace_bytes
    assert ws(0, 100, 4, 64, 128, 2, 1) == ws(2, 0, 4, 64, 128, 2, 1) == 0
    assert ws(2, 100, 4, 60, 128, 2, 1) == ws(2, 100, 4, 64, 128, 3, 1) == ws(2, 100, 4, 64, 128, 2, 7) == 0
    assert ws(2, 100, 4, 64, 128, 2, 0) > need


def test_delta_scan_bwd_refusals(lib, L):
    mid = dict(init=None, seq=None, st=FAKE, dy=FAKE, df=None)
    outs = dict(dq=FAKE, dk=FAKE, dv=FAKE, ddt=FAKE, dbeta=FAKE, dA=FAKE, db=None, di=None)

    def call(**over):
        kw = {**RULE, **SIZE, **END, **mid, **outs, **over}
        return lib.ssd_delta_scan_bwd(*(kw[k] for k in (*RULE, *mid, *outs, *SIZE, *END)), None)
    assert call(b=0) == call(l=0) == call(l=-1) == L.SSD_ERR_SHAPE
    _shared(lambda **kw: L.SSD_OK if kw.pop("last", 0) else call(**kw), L, dict(last=1))
    for name in ("dy", "dq", "dk", "dv", "ddt", "dbeta", "dA"):
        assert call(**{name: None}) == L.SSD_ERR_NULL, name
    for name in ("q", "k", "v", "dy", "dq", "dk", "dv", "init", "st", "df", "di"):
        assert call(**{name: FAKE + 8}) == L.SSD_ERR_ALIGN, name
    for name in ("dA", "db", "seq"):
        assert call(**{name: FAKE + 2}) == L.SSD_ERR_ALIGN, name
    need = [lib.ssd_delta_scan_bwd_workspace_bytes(2, 100, 4, 64, 128, 2, 1, s) for s in (0, 1)]
    assert need[0] > need[1] > 0
    assert call(wsb=need[1] - 1) == L.SSD_ERR_WORKSPACE
    assert call(st=None, wsb=need[1]) == L.SSD_ERR_WORKSPACE
    assert call(ws=FAKE + 128) == L.SSD_ERR_ALIGN
    assert lib.ssd_delta_scan_bwd_workspace_bytes(0, 100, 4, 64, 128, 2, 1, 1) == 0


def test_delta_step_refusals(lib, L):
    size = dict(b=2, h=4, p=64, n=128, g=2, io=1)

    def call(**over):
        kw = {**RULE, **size, "state": FAKE, "y": FAKE, **over}
        return lib.ssd_delta_step(kw["state"], *(kw[k] for k in (*RULE, "y", *size)), None)
    _shared(call, L, dict(b=0, v=None))
    assert call(state=None) == call(y=None) == L.SSD_ERR_NULL
    assert call(b=1 << 22) == L.SSD_ERR_UNSUPPORTED
    for bad in (dict(state=FAKE + 8), dict(v=FAKE + 4), dict(y=FAKE + 4), dict(v=FAKE + 8, io=0),
                dict(q=FAKE + 1), dict(k=FAKE + 2, io=0)):
        assert call(**bad) == L.SSD_ERR_ALIGN, bad


def test_layer_norm_refusals(lib, L):
    def call(**over):
        kw = dict(x=FAKE, r=FAKE, w=FAKE, b=FAKE, eps=1e-5, y=FAKE, s=FAKE, st=FAKE, rows=10,
                  dim=40, io=1)
        kw.update(over)
        return lib.ssd_layer_norm(*kw.values(), None)
    assert call(io=3) == L.SSD_ERR_UNSUPPORTED
    for bad in (dict(rows=-1), dict(dim=0), dict(dim=-3), dict(eps=-1e-9), dict(eps=math.nan)):
        assert call(**bad) == L.SSD_ERR_SHAPE, bad
    assert call(dim=(1 << 24) + 1) == L.SSD_ERR_UNSUPPORTED
    assert call(rows=1 << 36, dim=64) == L.SSD_ERR_UNSUPPORTED
    assert call(x=None) == call(y=None) == L.SSD_ERR_NULL
    assert call(r=None) == L.SSD_ERR_NULL  # a sum of nothing
    for name in ("x", "r", "y", "s"):
        assert call(**{name: FAKE + 1}) == L.SSD_ERR_ALIGN, name
        assert call(**{name: FAKE + 2}, io=0) == L.SSD_ERR_ALIGN, name
    for name in ("w", "b", "st"):
        assert call(**{name: FAKE + 2}) == L.SSD_ERR_ALIGN, name
    assert call(rows=0, x=None) == L.SSD_OK


def test_layer_norm_bwd_refusals(lib, L):
    def call(**over):
        kw = dict(dy=FAKE, x=FAKE, st=FAKE, w=FAKE, ds=FAKE, dx=FAKE, dw=FAKE, db=FAKE, rows=1000,
                  dim=40, io=1, ws=FAKE, wsb=1 << 40)
        kw.update(over)
        return lib.ssd_layer_norm_bwd(*kw.values(), None)
    assert call(io=3) == L.SSD_ERR_UNSUPPORTED
    assert call(rows=-1) == call(dim=0) == L.SSD_ERR_SHAPE
    assert call(dim=(1 << 24) + 1) == L.SSD_ERR_UNSUPPORTED
    assert call(dx=None, dw=None, db=None) == L.SSD_ERR_NULL
    assert call(dy=None) == call(x=None) == call(st=None) == L.SSD_ERR_NULL
    for name in ("dy", "x", "ds", "dx"):
        assert call(**{name: FAKE + 1}) == L.SSD_ERR_ALIGN, name
    for name in ("st", "w", "dw", "db"):
        assert call(**{name: FAKE + 2}) == L.SSD_ERR_ALIGN, name
    need = lib.ssd_layer_norm_bwd_workspace_bytes(1000, 40)
    assert need > 0
    assert call(wsb=need - 1) == call(ws=None) == L.SSD_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == L.SSD_ERR_ALIGN
    assert lib.ssd_layer_norm_bwd_workspace_bytes(1, 40) == 0      # one workgroup writes the sums
    assert lib.ssd_layer_norm_bwd_workspace_bytes(-1, 40) == 0
    assert call(rows=0, dw=None, db=None) == L.SSD_OK
