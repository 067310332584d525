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
