"""The copies of the products' operands into LDS, followed on the host: the
kernels' own arithmetic (csrc/ssd_copies.hpp), every slot of every step of every
tile, compiled with the host compiler."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mamba_ssd_chunked_chunk_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "ssd_copies.hpp"
using namespace ssd;

// An operand of `rows` tile rows and a contraction of `cont`, in `parts` parts.
template <int ES, bool TR, int BM> long check(int64_t rows, int64_t cont, int64_t parts) {
    typedef TileGeometry<ES, TR, BM> T;
    const int64_t unit = 16 / ES, ld = ((TR ? rows : cont) + unit - 1) / unit * unit;
    const int64_t bytes = (TR ? cont : rows) * ld * ES;
    const int64_t all = (cont + T::BK - 1) / T::BK, kper = (all + parts - 1) / parts * T::BK;
    long bad = 0;
    for (int64_t k0 = 0; k0 < cont; k0 += kper)
        for (int64_t m0 = 0; m0 < rows; m0 += BM) {
            const int64_t kEnd = k0 + kper < cont ? k0 + kper : cont;
            const int steps = (int)((kEnd - k0 + T::BK - 1) / T::BK);
            const CopySteps<ES, TR, BM> c(ld, m0, rows, k0, kEnd, steps);
            for (int s = 0; s < steps; ++s)
                for (int slot = 0; slot < T::BYTES / 16; ++slot) {
                    const bool fin = s == steps - 1;
                    const int64_t off = T::offset(slot, ld), at = c.first + s * c.stride + off;
                    const bool read = !(fin && c.masked(slot)) && off + 16 <= (fin ? c.last : c.bytes);
                    // what the slot is for: its first element's tile row and contraction
                    const int64_t r = slot / T::CH, q = T::chunk(slot) * T::EPC;
                    const int64_t m = m0 + (TR ? q : r), k = k0 + s * T::BK + (TR ? r : q);
                    const bool needed = m < rows && k < kEnd;
                    const int64_t want = (TR ? k * ld + m : m * ld + k) * ES;
                    if (read && (at < 0 || at + 16 > bytes)) ++bad;   // outside the operand
                    if (needed && (!read || at != want)) ++bad;       // or not what is needed
                    if (k >= kEnd && read) ++bad;                     // or not zero behind the end
                }
        }
    if (bad) printf("ES %d TR %d BM %d rows %ld cont %ld parts %ld: %ld\n", ES, TR, BM, (long)rows,
                    (long)cont, (long)parts, bad);
    return bad;
}

template <int ES, int BM> long both() {
    long bad = 0;
    const int64_t rows[] = {1, 4, 8, 16, 24, 31, 48, 63, 64, 65, 96, 128, 130, 192, 200, 257};
    const int64_t cont[] = {1, 8, 16, 17, 31, 32, 33, 63, 64, 65, 96, 128, 129, 191, 257, 300};
    for (int64_t r : rows)
        for (int64_t k : cont)
            for (int64_t p = 1; p <= 3; ++p) bad += check<ES, false, BM>(r, k, p) + check<ES, true, BM>(r, k, p);
    return bad;
}

int main() {
    const long bad = both<2, 64>() + both<2, 128>() + both<2, 192>() + both<4, 64>() + both<4, 128>();
    printf("%ld\n", bad);
    return bad != 0;
}
"""


def test_every_copy_stays_inside_its_operand_and_none_is_missing(tmp_path):
    src, exe = tmp_path / "copies.cpp", tmp_path / "copies"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout[-2000:]
