// Which bytes of an operand a product's workgroup copies into LDS: plain
// arithmetic without device code, so that a test on the host can follow every
// copy of the kernels.
#pragma once

#include <stdint.h>

namespace ssd {

// An operand's tile is ROWS stored rows of 16-byte chunks, CH chunks a row,
// chunk c of row r kept at slot c ^ f(r).
//   contraction contiguous: ROWS = tile rows m, a row is 128 bytes of k
//   contraction outermost:  ROWS = 128 / ES values of k, a row is the tile's m
// ES: bytes of an element.
template <int ES, bool TR, int BM> struct TileGeometry {
    static constexpr int EPC = 16 / ES;
    static constexpr int BK = 128 / ES;
    static constexpr int ROWS = TR ? BK : BM;
    static constexpr int CH = TR ? BM / EPC : 8;
    static constexpr int BYTES = ROWS * CH * 16;
    static_assert(!TR || (ES == 2 ? CH % 8 : CH % 16) == 0, "f stays inside a row");
    static constexpr int f(int r) {
        if (!TR) return r & 7;
        // The transposing loads of 32 lanes take 32 bytes of rows 0-3 and 8-11
        // (4-7 and 12-15): f moves them to eight different eighths of the banks.
        // Rows of an odd number of 128 bytes alternate halves by themselves.
        if (ES == 2)
            return CH % 16 == 0 ? ((r & 3) | ((r >> 1) & 4)) << 1 : (r & 2) | ((r >> 1) & 4);
        return ((r >> 2) & 3) << 2;  // fp32: 64 bytes of rows 4 apart
    }
    // The chunk of its row that lies at a slot of the tile, and where it is read:
    // bytes from the step's first element.
    static constexpr int chunk(int slot) { return slot % CH ^ f(slot / CH); }
    static constexpr uint32_t offset(int slot, int64_t ld) {
        return (uint32_t)(slot / CH * ld + chunk(slot) * EPC) * (uint32_t)ES;
    }
};

// The steps of one tile's copies.  Offsets are the same in every step; the first
// element moves on by `stride` bytes.  What lies past the operand's rows or its
// contraction is read as zeros: contraction contiguous, the reach ends with the
// rows (the chunks of a row past its end are masked in the last step);
// contraction outermost, it ends with the contraction.  There a row narrower
// than the tile runs on into the rows behind it, so the reach has to count in
// every step, not in the last one alone: the steps before the last end where
// the last but one does, which leaves them their own rows.  Offsets inside a tile
// stay below 2^30, so a reach is cut off at kOpen.
constexpr int64_t kOpen = 0x7fffffff;

template <int ES, bool TR, int BM> struct CopySteps {
    typedef TileGeometry<ES, TR, BM> T;
    int64_t first, stride;  // bytes: the operand's start to the first step, step to step
    int bytes, last;        // reach in a step, and in the last one
    int tail;               // contraction elements in the last step
    // Rows m0 .. of the operand (it has mEnd), `steps` steps from k0 to kEnd, `ld`
    // elements from one stored row to the next.
    constexpr CopySteps(int64_t ld, int64_t m0, int64_t mEnd, int64_t k0, int64_t kEnd, int steps)
        : first((TR ? k0 * ld + m0 : m0 * ld + k0) * ES), stride(TR ? T::BK * ld * ES : T::BK * ES),
          bytes(0), last(0), tail((int)(kEnd - (k0 + (int64_t)(steps - 1) * T::BK))) {
        const int64_t end = (TR ? tail * ld - m0 : (mEnd - m0) * ld) * ES;
        const int64_t each = TR ? end + stride : end;
        last = (int)(end < kOpen ? end : kOpen);
        bytes = (int)(each < kOpen ? each : kOpen);
    }
    // Whether the last step leaves a slot's chunk out.
    constexpr bool masked(int slot) const { return !TR && T::chunk(slot) * T::EPC >= tail; }
};

}  // namespace ssd
