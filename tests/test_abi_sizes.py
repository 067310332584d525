"""The sizes that ssd.h names as the limits of the linear layer and the gated
recurrence: taken up to them, refused beyond, before the HIP runtime is touched;
the queries return 0 beyond them.  Calls that pass the size checks end at a NULL
argument."""
import pytest

FAKE = 0x10000


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


def _up64(v):
    return (v + 63) // 64 * 64


# (rows, in, out): the last sizes below 2^34 values of rows rounded up to 64, and
# the first at it; widths at 2^20 and beyond
@pytest.mark.parametrize("m,k,n,ok", [
    ((1 << 28) - 1, 4, 4, True), (1 << 28, 4, 4, False), (1 << 28, 1, 64, False),
    ((1 << 27) - 1, 65, 8, True), (1 << 27, 65, 8, False), (1 << 27, 8, 65, False),
    (8, 1 << 20, (1 << 14) - 1, True), (8, 1 << 20, 1 << 14, False), (8, 8, 1 << 20, True),
    (8, (1 << 20) + 1, 8, False), (8, 8, (1 << 20) + 1, False), (1 << 31, 1, 1, False)])
def test_linear_limits(lib, L, m, k, n, ok):
    want = L.SSD_ERR_NULL if ok else L.SSD_ERR_UNSUPPORTED
    for io in (0, 1):
        assert lib.ssd_linear(None, FAKE, None, None, FAKE, None, 0, m, k, n, io, FAKE, 1 << 50,
                              None) == want
        assert lib.ssd_linear_bwd(None, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, m, k, n, io, FAKE,
                                  1 << 50, None) == want
        assert (lib.ssd_linear_bwd_workspace_bytes(m, k, n, 1, io) > 0) == ok
        if not ok:
            assert lib.ssd_linear_workspace_bytes(m, k, n, io) == 0
    if ok:  # the threads of one launch that lays x and the weight out again
        assert (m + n) * _up64(k) // 8 + 512 <= 1 << 32


@pytest.mark.parametrize("b,l,d,ok", [
    (65535, 64, 64, True), (65536, 64, 64, False), (1, 1 << 28, 64, True), (1, (1 << 28) + 1, 64, False),
    (1, 64, 1 << 24, True), (1, 64, (1 << 24) + 1, False), (2, 64 * 255, 64 * 16448, True),
    (2, 64 * 256, 64 * 16384, False), (1, 64 * 8191 + 1, 64 * 1024, False)])
def test_gated_scan_limits(lib, L, b, l, d, ok):
    want = L.SSD_ERR_NULL if ok else L.SSD_ERR_UNSUPPORTED
    assert ok == (b <= 65535 and l <= 1 << 28 and d <= 1 << 24
                  and b * -(-d // 64) * -(-l // 64) < 1 << 23)
    for io in (0, 1):
        assert lib.ssd_gated_scan(None, FAKE, FAKE, 8.0, None, None, FAKE, None, None, b, l, d, io,
                                  FAKE, 1 << 50, None) == want
        assert lib.ssd_gated_scan_bwd(None, FAKE, FAKE, 8.0, None, None, None, FAKE, None, FAKE,
                                      FAKE, FAKE, None, b, l, d, io, FAKE, 1 << 50, None) == want
    assert (lib.ssd_gated_scan_workspace_bytes(b, l, d) > 0) == ok
    assert (lib.ssd_gated_scan_bwd_workspace_bytes(b, l, d) > 0) == ok


@pytest.mark.parametrize("b,d,ok", [(1, 1 << 24, True), (1, (1 << 24) + 1, False),
                                    ((1 << 31), 1, True), ((1 << 31) + 1, 1, False),
                                    ((1 << 32) - 256, 1, False), ((1 << 24) - 1, 256, True),
                                    ((1 << 24) + 1, 255, True), (1 << 31, 3, False)])
def test_gated_step_limits(lib, L, b, d, ok):
    """No product of batch and dim above 2^32 - 256 channels one at a time is taken;
    wider accesses take as many times more."""
    want = L.SSD_ERR_NULL if ok else L.SSD_ERR_UNSUPPORTED
    for io in (0, 1):
        if want == L.SSD_ERR_NULL:
            assert lib.ssd_gated_step(None, FAKE, FAKE, FAKE, 8.0, FAKE, b, d, io, None) == want
        else:  # the count of threads is checked behind the pointers; one channel a lane
            off = FAKE + (4 if io == 0 else 2)
            assert lib.ssd_gated_step(FAKE + 4, off, off, FAKE + 4, 8.0, off, b, d, io, None) == want


def test_workspace_queries_know_their_types(lib):
    """The binding's queries take the names "f32" and "bf16" as state_chunks does,
    and no other for one of them."""
    import mamba_ssd_chunked_chunk_amd as ssd
    assert ssd.linear_workspace_bytes(300, 65, 40, io="bf16") == \
        lib.ssd_linear_workspace_bytes(300, 65, 40, 1)
    assert ssd.linear_workspace_bytes(300, 65, 40, io="f32") == \
        lib.ssd_linear_workspace_bytes(300, 65, 40, 0)
    assert ssd.linear_bwd_workspace_bytes(300, 65, 40, "silu", io="f32") == \
        lib.ssd_linear_bwd_workspace_bytes(300, 65, 40, 1, 0)
    for name in ("bfloat16", "f16", None):
        with pytest.raises(ValueError, match="io"):
            ssd.linear_workspace_bytes(300, 65, 40, io=name)
        with pytest.raises(ValueError, match="io"):
            ssd.linear_bwd_workspace_bytes(300, 65, 40, io=name)
