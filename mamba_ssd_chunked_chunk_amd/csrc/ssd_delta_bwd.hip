// The gated delta rule's gradient (formulas in ssd_delta.hpp), from the states
// in front of the chunks:
//
// k_delta_mid, all chunks in parallel: N = v - P^T k of 16 value columns per
// wave, and what else does not need the adjoint state.  Bound by memory: 4 x 2048
// tokens of 16 heads of 128 x 128 move 0.69 GB in 130 us.
//
// k_delta_rev, chunk after chunk from the end: the adjoint state of 16 value
// columns in a wave's registers, as in the forward pass; leaves Z, dV, the
// adjoint state behind every chunk, and per token the terms of the decays'
// gradient that reach into the chunk from outside.  What k_delta_mid left, and
// the state in front, come into registers a chunk ahead.  Bound by memory and the
// chain of one wave, 1900 instructions a chunk, about alike: 205 us and 0.71 GB
// for the same call, 6.4 us a chunk.
//
// k_delta_grad, all chunks in parallel: dq and dk, which contract over the value
// columns, and the decays' terms inside the chunk.  A wave owns 16 tokens, all
// keys of them in registers, transposed ([key][token]), so that the masked
// products dY U^T and Z N^T are the next product's operands as they stand; the
// heads that share q and k are walked in order by one workgroup.  With bf16 io
// its operands are two fp16 terms, and a step of its products takes both of 16 value
// columns for the two halves of an instruction's contraction.  178 us for the same
// call, 0.59 GB (121 us of a copy).
#include "ssd_delta.hpp"

#include <math.h>

#include "../../include/ssd.h"

namespace ssd {

namespace {

// A matrix of 16 value columns as k_delta_grad's operand: fragment f of it.
template <typename IO, int PL>
__device__ __forceinline__ void put_operand(typename GradOp<IO>::type *dst, const f32x4 &a, const f32x4 &b,
                                            const Split &s, int f, int plane, int lane) {
    if constexpr (sizeof(IO) == 2) {
        *reinterpret_cast<f16x8 *>(dst + f * 512 + lane * 8) = s.hi;
        if constexpr (PL == 2) *reinterpret_cast<f16x8 *>(dst + plane + f * 512 + lane * 8) = s.lo;
    } else {
        *reinterpret_cast<f32x4 *>(dst + f * 512 + lane * 8) = a;
        *reinterpret_cast<f32x4 *>(dst + f * 512 + lane * 8 + 4) = b;
    }
}
// Elements of N or Z, and of a state, of 16 columns of a chunk.
template <typename IO> constexpr int kOperandN = GradOp<IO>::PL * 2 * 512;
template <typename IO, int N> constexpr int kOperandS = GradOp<IO>::PL * (N / 32) * 512;

// The transposed product of a lower triangle (its hi and lo images at M) with
// the rows in f: row tile jt.
__device__ __forceinline__ f32x4 tri_t(const f16 *M, int jt, const Split *f, int lane) {
    f32x4 t = zero4();
#pragma unroll
    for (int tb = jt >> 1; tb < 2; ++tb) {
        const int p0 = tri_piece(2 * tb, jt >> 1), p1 = tri_piece(2 * tb + 1, jt >> 1);
        const f16x8 h = img_cols(M, p0, p1, jt, lane);
        t = mma16(h, f[tb].hi, t);
        t = mma16(h, f[tb].lo, t);
        t = mma16(img_cols(M + kPieces * 512, p0, p1, jt, lane), f[tb].hi, t);
    }
    return t;
}

template <typename IO, int N>
__global__ __launch_bounds__(256, 2) void k_delta_mid(DeltaArgs a) {
    typedef FwdBuf<IO, N, true> B;
    typedef typename GradOp<IO>::type OT;
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int XB = N / 32, NT = N / 16, IMG = kDC * N;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int g = lane >> 4, j16 = lane & 15;
    const int cols = 16 * nw, slices = a.p / cols, cts = a.p >> 4;
    int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int col0 = (int)(item % slices) * cols;
    item /= slices;
    const int64_t hh = item % a.h, ci = item / a.h, c = ci % a.nc, bb = ci / a.nc, hi = ci * a.h + hh;
    const int col = col0 + 16 * wave, ct = col >> 4;

    FwdSrc<IO, N, true> src(a, bb, c, hh, col0, cols);
    src.copy(lds_address(lds), wave, nw, lane);
    f32x4 S[NT];
    {
        const float *s0 = c ? a.kept + (hi - a.h) * N * a.p
                            : a.init ? a.init + (bb * a.h + hh) * N * a.p : nullptr;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            S[x] = zero4();
            if (s0)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[x][r] = s0[(16 * x + 4 * g + r) * a.p + col + j16];
        }
    }
    vm_wait<0>();
    lds_barrier();
    const f16 *K = reinterpret_cast<const f16 *>(lds + B::K);
    const f16 *Q = reinterpret_cast<const f16 *>(lds + B::Q);
    const f16 *T = reinterpret_cast<const f16 *>(lds + B::T);
    const f16 *P = reinterpret_cast<const f16 *>(lds + B::P);
    const float *rows = reinterpret_cast<const float *>(lds + B::R);
    const IO *V = reinterpret_cast<const IO *>(lds + B::V);
    const IO *dY = V + kDC * cols;
    float *scales = a.scales + (hi * cts + ct) * kScales;

    float mx = 0.f;
#pragma unroll
    for (int x = 0; x < NT; ++x) mx = abs_max(mx, S[x]);
    const Pow2 ps(tile_max(mx));
    Split sf[XB];
    OT *simg = static_cast<OT *>(a.simg) + (hi * cts + ct) * kOperandS<IO, N>;
#pragma unroll
    for (int kb = 0; kb < XB; ++kb) {
        sf[kb] = split8(S[2 * kb], S[2 * kb + 1], ps.sc);
        put_operand<IO, 2>(simg, S[2 * kb], S[2 * kb + 1], sf[kb], kb, XB * 512, lane);
    }
    f32x4 R[4];
    f32x4 *g0 = reinterpret_cast<f32x4 *>(a.g0 + (hi * cts + ct) * (16 * kDC)) + lane;
    float *qs = a.toks + ((hi * cts + ct) * kSums + kSumQ) * kDC;
    mx = 0.f;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        f32x4 t = zero4(), u = zero4();
#pragma unroll
        for (int kb = 0; kb < XB; ++kb) {
            const f16x8 k = img_rows(K, rt * XB + kb, lane), q = img_rows(Q, rt * XB + kb, lane);
            t = mma16(k, sf[kb].hi, t);
            u = mma16(q, sf[kb].hi, u);
            t = mma16(k, sf[kb].lo, t);
            u = mma16(q, sf[kb].lo, u);
            if constexpr (F32) {
                t = mma16(img_rows(K + IMG, rt * XB + kb, lane), sf[kb].hi, t);
                u = mma16(img_rows(Q + IMG, rt * XB + kb, lane), sf[kb].hi, u);
            }
        }
        const f32x4 v = lds_tile(V, cols, rt, 16 * wave, lane), f = row4(rows, kReadK, rt, lane);
        const f32x4 d = lds_tile(dY, cols, rt, 16 * wave, lane), fq = row4(rows, kReadQ, rt, lane);
        f32x4 s;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            t[r] *= f[r] * ps.inv;
            R[rt][r] = v[r] - t[r];
            s[r] = sum16(d[r] * (fq[r] * ps.inv * u[r]));
        }
        g0[64 * rt] = t;
        if (j16 == 0) *reinterpret_cast<f32x4 *>(qs + 16 * rt + 4 * g) = s;
        mx = abs_max(mx, R[rt]);
    }
    const Pow2 pr(col_max(mx));
    Split rf[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) rf[tb] = split8(R[2 * tb], R[2 * tb + 1], pr.sc);
    const float undo = pr.inv * rows[kCarry * kDC + kInvT];
    mx = 0.f;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        f32x4 t = zero4();
#pragma unroll
        for (int tb = 0; tb <= rt / 2; ++tb) {
            const int p0 = tri_piece_t(2 * tb, rt >> 1), p1 = tri_piece_t(2 * tb + 1, rt >> 1);
            const f16x8 th = img_cols(T, p0, p1, rt, lane);
            t = mma16(th, rf[tb].hi, t);
            t = mma16(th, rf[tb].lo, t);
            t = mma16(img_cols(T + kPieces * 512, p0, p1, rt, lane), rf[tb].hi, t);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) R[rt][r] = t[r] * undo;
        mx = abs_max(mx, R[rt]);
    }
    const Pow2 pn(tile_max(mx));
    OT *nimg = static_cast<OT *>(a.nimg) + (hi * cts + ct) * kOperandN<IO>;
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
        put_operand<IO, 2>(nimg, R[2 * tb], R[2 * tb + 1], split8(R[2 * tb], R[2 * tb + 1], pn.sc), tb,
                           1024, lane);
    // dY as k_delta_grad's operand, and scale tril(Q K^T)^T dY
    float my = 0.f;
    mx = 0.f;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        const f32x4 d = lds_tile(dY, cols, rt, 16 * wave, lane), f = row4(rows, kFq, rt, lane);
#pragma unroll
        for (int r = 0; r < 4; ++r) R[rt][r] = d[r] * f[r];
        mx = abs_max(mx, R[rt]);
        my = abs_max(my, d);
    }
    const Pow2 pe(col_max(mx)), py(tile_max(my));
    OT *yimg = static_cast<OT *>(a.yimg) + (hi * cts + ct) * 1024;
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
        rf[tb] = split8(R[2 * tb], R[2 * tb + 1], pe.sc);
        const f32x4 d0 = lds_tile(dY, cols, 2 * tb, 16 * wave, lane),
                    d1 = lds_tile(dY, cols, 2 * tb + 1, 16 * wave, lane);
        put_operand<IO, 1>(yimg, d0, d1, split8(d0, d1, py.sc), tb, 0, lane);
    }
    f32x4 *x0 = reinterpret_cast<f32x4 *>(a.x0 + (hi * cts + ct) * (16 * kDC)) + lane;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        f32x4 t = tri_t(P, rt, rf, lane);
        const f32x4 fk = row4(rows, kFk, rt, lane);
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] *= fk[r] * pe.inv;
        x0[64 * rt] = t;
    }
    if (lane == 0) scales[kScS] = ps.inv, scales[kScN] = pn.inv, scales[kScY] = py.inv;
}

template <typename IO, int N> struct RevBuf {
    typedef GroupImg<IO, N> G;
    typedef HeadImg<true> H;
    static constexpr int ROWS = H::P - H::R, INV = H::BYTES - H::M;
    static constexpr int K = 0, Q = G::Q, R = G::BYTES, M = R + ROWS, DY = M + INV;
    static __host__ __device__ int bytes(int cols) { return DY + kDC * cols * (int)sizeof(IO); }
};

// Where a chunk's operands of one head and `cols` columns are; back() moves to
// the chunk in front.
template <typename IO, int N> struct RevSrc {
    typedef RevBuf<IO, N> B;
    const char *grp, *head, *dy;
    int64_t sg, sh, sy;
    uint32_t pitch;
    int rb, len;
    __device__ RevSrc(const DeltaArgs &a, int64_t bb, int64_t hh, int col0, int cols) {
        const int64_t ci = bb * a.nc + a.nc - 1, t0 = (a.nc - 1) * kDC;
        grp = uni(a.gimg + (ci * a.g + hh / (a.h / a.g)) * B::G::BYTES);
        head = uni(a.himg + (ci * a.h + hh) * a.hstride);
        const int64_t at = (((bb * a.l + t0) * a.h + hh) * a.p + col0) * (int64_t)sizeof(IO);
        dy = uni(static_cast<const char *>(a.dy) + at);
        pitch = (uint32_t)(a.h * a.p * sizeof(IO));
        sg = a.g * B::G::BYTES, sh = a.h * a.hstride, sy = (int64_t)kDC * pitch;
        rb = cols * (int)sizeof(IO), len = uni((int)(a.l - t0));
    }
    __device__ void back() { grp -= sg, head -= sh, dy -= sy, len = kDC; }
    __device__ void copy(uint32_t buf, int wave, int nw, int lane) const {
        copy_image<B::G::BYTES>(grp, buf, wave, nw, lane);
        copy_image<B::ROWS>(head + B::H::R, buf + B::R, wave, nw, lane);
        copy_image<B::INV>(head + B::H::M, buf + B::M, wave, nw, lane);
        copy_rows(dy, pitch, rb, len, buf + B::DY, wave, nw, lane);
    }
};

// tri_t of an inverse, which is kept transposed.
__device__ __forceinline__ f32x4 inv_t(const f16 *M, int jt, const Split *f, int lane) {
    f32x4 t = zero4();
#pragma unroll
    for (int ib = jt >> 1; ib < 2; ++ib) {
        const f16x8 h = img_rows(M, tri_piece_t(jt, ib), lane);
        t = mma16(h, f[ib].hi, t);
        t = mma16(h, f[ib].lo, t);
        t = mma16(img_rows(M + kPieces * 512, tri_piece_t(jt, ib), lane), f[ib].hi, t);
    }
    return t;
}

// What k_delta_mid left of a chunk's 16 columns, and the state in front of it, in
// registers a chunk ahead; each part is loaded where the one before was used.
template <typename IO, int N> struct RevAhead {
    typedef typename GradOp<IO>::type OT;
    static constexpr bool F32 = sizeof(IO) == 4;
    static constexpr int NT = N / 16;
    f32x4 S[NT], g0[4], x0[4], n[F32 ? 4 : 1];
    f16x8 nh[F32 ? 1 : 2], nl[F32 ? 1 : 2];
    float ninv;
    __device__ void load_state(const DeltaArgs &a, int64_t bb, int64_t hh, int64_t c, int col, int lane) {
        const float *s0 = c ? a.kept + ((bb * a.nc + c - 1) * a.h + hh) * N * a.p
                            : a.init ? a.init + (bb * a.h + hh) * N * a.p : nullptr;
        // without a state in front all of it lies beyond the resource and comes as zeros
        const Rsrc rs = make_rsrc(reinterpret_cast<const float *>(uni(s0)), s0 ? N * a.p * 4 : 0);
        const int row = 4 * a.p, off = (4 * (lane >> 4) * a.p + col + (lane & 15)) * 4;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[x][r] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, (16 * x + r) * row, 0));
    }
    __device__ void load_x(const DeltaArgs &a, int64_t at, int lane) {
        const f32x4 *x = reinterpret_cast<const f32x4 *>(a.x0 + at * (16 * kDC)) + lane;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) x0[rt] = x[64 * rt];
    }
    __device__ void load_n(const DeltaArgs &a, int64_t at, int lane) {
        const f32x4 *k = reinterpret_cast<const f32x4 *>(a.g0 + at * (16 * kDC)) + lane;
        const OT *v = static_cast<const OT *>(a.nimg) + at * kOperandN<IO> + lane * 8;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) g0[rt] = k[64 * rt];
        if constexpr (F32) {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
                n[rt] = *reinterpret_cast<const f32x4 *>(v + 512 * (rt >> 1) + 4 * (rt & 1));
        } else {
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                nh[tb] = *reinterpret_cast<const f16x8 *>(v + 512 * tb);
                nl[tb] = *reinterpret_cast<const f16x8 *>(v + 1024 + 512 * tb);
            }
            ninv = a.scales[at * kScales + kScN];
        }
    }
    __device__ void wait() {
        landed(S), landed(g0), landed(x0);
        if constexpr (F32) {
            landed(n);
        } else {
            landed(nh), landed(nl);
            asm volatile("" : "+v"(ninv));
        }
    }
    __device__ f32x4 rows_n(int rt) const {
        if constexpr (F32) {
            return n[rt];
        } else {
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const f16 h = nh[rt >> 1][4 * (rt & 1) + r], l = nl[rt >> 1][4 * (rt & 1) + r];
                v[r] = ((float)h + (float)l) * ninv;
            }
            return v;
        }
    }
};

template <typename IO, int N, int NB>
__global__ __launch_bounds__(256, 1) void k_delta_rev(DeltaArgs a) {
    typedef RevBuf<IO, N> B;
    typedef typename GradOp<IO>::type OT;
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int XB = N / 32, NT = N / 16, IMG = kDC * N;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int g = lane >> 4, j16 = lane & 15;
    const int cols = 16 * nw, slices = a.p / cols;
    int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int col0 = (int)(item % slices) * cols;
    item /= slices;
    const int64_t hh = item % a.h, bb = item / a.h;
    const int col = col0 + 16 * wave, ct = col >> 4, cts = a.p >> 4;
    const int bufbytes = B::bytes(cols);
    const uint32_t base = lds_address(lds);
    const uint32_t pitch = (uint32_t)(a.h * a.p * sizeof(IO));

    RevSrc<IO, N> src(a, bb, hh, col0, cols);
    src.copy(base + (NB == 2 ? ((a.nc - 1) & 1) * bufbytes : 0), wave, nw, lane);
    f32x4 dS[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        dS[x] = zero4();
        if (a.dfin)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dS[x][r] = a.dfin[((bb * a.h + hh) * N + 16 * x + 4 * g + r) * a.p + col + j16];
    }
    landed(dS);
    // tiles of the chunk in front are `step` further back
    const int64_t step = a.h * cts;
    RevAhead<IO, N> in;
    {
        const int64_t at = ((bb * a.nc + a.nc - 1) * a.h + hh) * cts + ct;
        in.load_state(a, bb, hh, a.nc - 1, col, lane);
        in.load_x(a, at, lane);
        in.load_n(a, at, lane);
    }
    for (int64_t c = a.nc - 1; c >= 0; --c) {
        const char *buf = lds + (NB == 2 ? (c & 1) * bufbytes : 0);
        // the copies of this chunk are older than the last chunk's stores (these at
        // the least: dV, the operands and the tokens' sums)
        if (c == a.nc - 1 || NB == 1)
            vm_wait<0>();
        else
            vm_wait<16 + 2 * XB + 4 + 12>();
        in.wait();
        lds_barrier();
        const int64_t hi = (bb * a.nc + c) * a.h + hh, t0 = c * kDC, at = hi * cts + ct;
        // the chunk in front, or once more the first, whose values are not used then
        const int64_t front = c ? c - 1 : 0, ahead = c ? at - step : at;
        const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
        if (NB == 2 && c > 0) {
            src.back();
            src.copy(base + ((c - 1) & 1) * bufbytes, wave, nw, lane);
        }
        const f16 *K = reinterpret_cast<const f16 *>(buf + B::K);
        const f16 *Q = reinterpret_cast<const f16 *>(buf + B::Q);
        const f16 *M = reinterpret_cast<const f16 *>(buf + B::M);
        const float *rows = reinterpret_cast<const float *>(buf + B::R);
        const IO *dY = reinterpret_cast<const IO *>(buf + B::DY);
        const float carry = rows[kCarry * kDC + kKeep];

        // e^{G_C} <S, dS> of these columns
        {
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) s = fmaf(in.S[x][r], dS[x][r], s);
            s = sum16(s);
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (lane == 0) a.eend[at] = carry * s;
            in.load_state(a, bb, hh, front, col, lane);
        }
        // the adjoint state behind the chunk: split, and kept for k_delta_grad
        float mx = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) mx = abs_max(mx, dS[x]);
        const Pow2 ps(tile_max(mx));
        Split sf[XB];
        OT *ds = static_cast<OT *>(a.dsimg) + at * kOperandS<IO, N>;
#pragma unroll
        for (int kb = 0; kb < XB; ++kb) {
            sf[kb] = split8(dS[2 * kb], dS[2 * kb + 1], ps.sc);
            put_operand<IO, 2>(ds, dS[2 * kb], dS[2 * kb + 1], sf[kb], kb, XB * 512, lane);
        }
        // scale e^G dY
        f32x4 G[4];
        mx = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 d = lds_tile(dY, cols, rt, 16 * wave, lane), f = row4(rows, kReadQ, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) G[rt][r] = d[r] * f[r];
            mx = abs_max(mx, G[rt]);
        }
        const Pow2 pe(col_max(mx));
        Split gf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) gf[tb] = split8(G[2 * tb], G[2 * tb + 1], pe.sc);
        // dU = tril(Q K^T)^T dY + e^{G_C - G} K dS
        f32x4 U[4], KD[4];
        mx = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            f32x4 t = zero4();
#pragma unroll
            for (int kb = 0; kb < XB; ++kb) {
                const f16x8 k = img_rows(K, rt * XB + kb, lane);
                t = mma16(k, sf[kb].hi, t);
                t = mma16(k, sf[kb].lo, t);
                if constexpr (F32) t = mma16(img_rows(K + IMG, rt * XB + kb, lane), sf[kb].hi, t);
            }
            const f32x4 wk = row4(rows, kWriteK, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                KD[rt][r] = wk[r] * ps.inv * t[r];
                U[rt][r] = in.x0[rt][r] + KD[rt][r];
            }
            mx = abs_max(mx, U[rt]);
        }
        in.load_x(a, ahead, lane);
        // Z, dV = beta Z, and their rows' products
        const Pow2 pu(col_max(mx));
        const float undo = pu.inv * rows[kCarry * kDC + kInvM];
        Split uf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) uf[tb] = split8(U[2 * tb], U[2 * tb + 1], pu.sc);
        f32x4 Z[4], W[4];
        mx = 0.f;
        float mz = 0.f;
        const Rsrc rv = make_rsrc(static_cast<IO *>(a.dv) + ((bb * a.l + t0) * a.h + hh) * a.p + col,
                                  (int64_t)(len - 1) * pitch + 16 * sizeof(IO));
        float *toks = a.toks + (at * kSums) * kDC;
        float *scales = a.scales + at * kScales;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 t = inv_t(M, rt, uf, lane), be = row4(rows, kBeta, rt, lane),
                        rk = row4(rows, kReadK, rt, lane), gk = in.g0[rt], n = in.rows_n(rt);
            f32x4 sk, so, sz;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                Z[rt][r] = t[r] * undo;
                const float v = be[r] * Z[rt][r];
                W[rt][r] = rk[r] * v;
                buf_put(rv, (16 * rt + 4 * g + r) * pitch + j16 * sizeof(IO), v, IO{});
                sk[r] = sum16(v * gk[r]);
                so[r] = sum16(be[r] * n[r] * KD[rt][r]);
                sz[r] = sum16(Z[rt][r] * n[r]);
            }
            mx = abs_max(mx, W[rt]);
            mz = abs_max(mz, Z[rt]);
            if (j16 == 0) {
                float *o = toks + 16 * rt + 4 * g;
                *reinterpret_cast<f32x4 *>(o + kSumK * kDC) = sk;
                *reinterpret_cast<f32x4 *>(o + kSumOut * kDC) = so;
                *reinterpret_cast<f32x4 *>(o + kSumZ * kDC) = sz;
            }
        }
        in.load_n(a, ahead, lane);
        const Pow2 pz(tile_max(mz));
        OT *dz = static_cast<OT *>(a.zimg) + at * kOperandN<IO>;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
            put_operand<IO, 2>(dz, Z[2 * tb], Z[2 * tb + 1], split8(Z[2 * tb], Z[2 * tb + 1], pz.sc), tb,
                               1024, lane);
        if (lane == 0) scales[kScD] = ps.inv, scales[kScZ] = pz.inv;
        // dS <- e^{G_C} dS + Q^T (scale e^G dY) - K^T (e^G dV)
        const Pow2 pw(col_max(mx));
        Split wf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) wf[tb] = split8(W[2 * tb], W[2 * tb + 1], pw.sc);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            f32x4 t = zero4(), u = zero4();
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const int p0 = 2 * tb * XB + (x >> 1), p1 = p0 + XB;
                const f16x8 q = img_cols(Q, p0, p1, x, lane), k = img_cols(K, p0, p1, x, lane);
                t = mma16(q, gf[tb].hi, t);
                t = mma16(q, gf[tb].lo, t);
                u = mma16(k, wf[tb].hi, u);
                u = mma16(k, wf[tb].lo, u);
                if constexpr (F32) {
                    t = mma16(img_cols(Q + IMG, p0, p1, x, lane), gf[tb].hi, t);
                    u = mma16(img_cols(K + IMG, p0, p1, x, lane), wf[tb].hi, u);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dS[x][r] = fmaf(carry, dS[x][r], fmaf(t[r], pe.inv, -pw.inv * u[r]));
        }
        if (NB == 1 && c > 0) {
            lds_barrier();  // everyone is done with the buffer
            src.back();
            src.copy(base, wave, nw, lane);
        }
    }
    if (a.dinit) {
        float *dst = a.dinit + (bb * a.h + hh) * N * a.p + col + j16;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(16 * x + 4 * g + r) * a.p] = dS[x][r];
    }
}

// ------------------------------------------------------------- dq and dk ---
typedef Frag8<float>::type f32x8;
__device__ __forceinline__ f32x4 mma8(f16x8 a, f16x8 b, f32x4 c) { return mma16(a, b, c); }
__device__ __forceinline__ f32x4 mma8(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = Mfma<float>::mma(a[e], b[e], c);
    return c;
}

// Keeps the operands of later steps from being read ahead of the registers.
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// Rows in memory come into LDS in the order of memory: pieces of 16 rows x 32
// columns whose lane (t & 15) + 16 ((x >> 3) & 3) holds the eight elements from
// x & ~7 on (an operand fragment contracted over x in that order, lane group g
// the eight indices 8 g ..).  Images contracted over their rows are then read in
// the same order.
// p0 is the piece of the first 16 rows, `next` pieces further that of the others.
template <typename IO>
__device__ __forceinline__ typename Frag8<IO>::type cols_nat(const IO *img, int p0, int next, int x16,
                                                            int lane) {
    const int g = lane >> 4, j = lane & 15;
    const IO *a = img + (g >> 1) * next * 512 + 64 * (g & 1) + p0 * 512 + 4 * (x16 & 1);
    if constexpr (sizeof(IO) == 2) {
        a += ((j >> 2) + 16 * (j & 3)) * 8;
        const f16x4 u = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)a));
        const f16x4 w = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)(a + 32)));
        return __builtin_bit_cast(typename Frag8<IO>::type,
                                  f16x8{u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]});
    } else {
        a += 128 * (j >> 2) + (j & 3);
        typename Frag8<IO>::type r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = a[8 * e];
        return r;
    }
}

// 64 rows, W valid columns of 32 XB, `pitch` elements apart, as such pieces.
template <int XB, typename IO>
__device__ __forceinline__ void copy_nat(const IO *src, int64_t pitch, int W, int len, uint32_t dst,
                                         int wave, int lane) {
    constexpr int PER = sizeof(IO) / 2;  // copies of 1024 bytes in a piece
    const RsrcW r = make_rsrc_w(src, ((int64_t)(len - 1) * pitch + W) * (int64_t)sizeof(IO));
    for (int i = wave; i < 4 * XB * PER; i += 4) {
        const int piece = i / PER, part = (i % PER) * 64 + lane, ln = part / PER;
        const int row = 16 * (piece / XB) + (ln & 15);
        const int x = 32 * (piece % XB) + 8 * (ln >> 4) + (PER == 2 ? 4 * (part & 1) : 0);
        const uint32_t off =
            row < len && x < W ? (uint32_t)((row * pitch + x) * (int64_t)sizeof(IO)) : 0xf0000000u;
        lds_dma16_at(r, dst + (i << 10), off, 0);
    }
}
// Fragment with x free (tile x16) and the 32 rows of the pieces' row tiles r0,
// r0 + 1 contracted, in the accumulators' order.
template <int XB, typename IO>
__device__ __forceinline__ typename Frag8<IO>::type nat_cols(const IO *img, int r0, int x16,
                                                            int lane) {
    const int g = lane >> 4, j = lane & 15, p0 = r0 * XB + (x16 >> 1), p1 = p0 + XB;
    if constexpr (sizeof(IO) == 2) {
        const int o = (4 * g + (j >> 2) + 16 * (2 * (x16 & 1) + ((j >> 1) & 1))) * 8 + 4 * (j & 1);
        const f16x4 u = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)(img + p0 * 512 + o)));
        const f16x4 w = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)(img + p1 * 512 + o)));
        return __builtin_bit_cast(typename Frag8<IO>::type,
                                  f16x8{u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]});
    } else {
        typename Frag8<IO>::type r;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = img[(e < 4 ? p0 : p1) * 512 +
                       (4 * g + (e & 3) + 16 * (2 * (x16 & 1) + (j >> 3))) * 8 + (j & 7)];
        return r;
    }
}
// Four elements (row, x .. x + 3) of such pieces.
template <int XB, typename IO>
__device__ __forceinline__ f32x4 nat4(const IO *img, int row, int x) {
    return ld4<IO>(img + ((row >> 4) * XB + (x >> 5)) * 512 +
                   ((row & 15) + 16 * ((x >> 3) & 3)) * 8 + (x & 4));
}

// A token's gradient through the normalisation (k[x] of its rows as the call has
// them, r is 1 / norm), and out: four keys per lane and tile.
template <int NT, typename IO, typename F>
__device__ __forceinline__ void put_rows(f32x4 (&d)[NT], F unit, IO *out, float r, int norm, bool live,
                                         int g) {
    if (norm) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const f32x4 v = unit(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fmaf(d[x][i], v[i], s);
        }
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const f32x4 v = unit(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[x][i] = r * fmaf(-s, v[i], d[x][i]);
        }
    }
    if (live)
#pragma unroll
        for (int x = 0; x < NT; ++x) st4<IO>(out + 16 * x + 4 * g, d[x]);
}

// Sum over the 16 lanes of a row of lanes, in fp64.
template <int CTRL> __device__ __forceinline__ double dpp_addd(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum16(double v) {
    v = dpp_addd<0x128>(v);
    v = dpp_addd<0x124>(v);
    v = dpp_addd<0x122>(v);
    return dpp_addd<0x121>(v);
}

// What undoes the powers of two of two operands, given by their inverses: two factors,
// as the inverses' product can leave fp32's range where the result does not.
struct Undo {
    float a, b;
    __device__ Undo(const float *s, int x, int y) {
        const auto of = [&](int i) { return (int)(__builtin_bit_cast(uint32_t, s[i]) >> 23); };
        const int e = of(x) + of(y) - 254, h = e / 2;
        a = ldexpf(1.f, h), b = ldexpf(1.f, e - h);
    }
};

// One stage of k_delta_grad in LDS: 16 value columns of a head in two terms, or 32 in
// fp32 (states in front and adjoint states behind as [column][key] images, N, Z and dY
// as [column][token]), or its group's k and q with the head's row arrays.
template <typename IO, int N> struct GradBuf {
    typedef GradOp<IO> O;
    static constexpr int E = (int)sizeof(typename O::type), TILES = 2 / O::PL;
    static constexpr int ST = N * 32 * E, TOK = kDC * 32 * E, TOKY = TOK / O::PL;
    static constexpr int S = 0, D = S + ST, NV = D + ST, Z = NV + TOK;
    static constexpr int DY = Z + TOK, SC = DY + TOKY, END1 = SC + (E == 2 ? 1024 : 0);
    static constexpr int K = 0, Q = K + kDC * N * E, R = Q + kDC * N * E;
    static constexpr int R2 = R + kRows * kDC * 4, END2 = R2 + kRowsGrad * kDC * 4;
    static constexpr int BYTES = END1 > END2 ? END1 : END2;
    // behind both buffers: row arrays for all stages of a head
    static constexpr int R0 = 2 * BYTES, BETA = R0 + kRowsGrad * kDC * 4, ALL = BETA + 1024;
};

template <typename IO, int N>
__global__ __launch_bounds__(256, 2) void k_delta_grad(DeltaArgs a) {
    typedef typename GradOp<IO>::type OT;
    typedef typename Frag8<OT>::type F;
    typedef GradBuf<IO, N> B;
    typedef HeadImg<true> H;
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int XB = N / 32, NT = N / 16;
    // an operand's second half in LDS: its low terms (of dY the same ones), or the next tile
    constexpr int NEXT = 2, NEXTY = F32 ? 2 : 0;
    __shared__ __align__(1024) char lds[B::ALL];

    const int w = wave_id(), own = threadIdx.x & 63;
    const int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int64_t gg = item % a.g, ci = item / a.g, c = ci % a.nc, bb = ci / a.nc;
    const int ratio = (int)(a.h / a.g);
    const int64_t t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
    const int cts = a.p >> 4;
    const uint32_t base = lds_address(lds);
    const int slices = (cts + B::TILES - 1) / B::TILES;
    const int64_t kq = ((bb * a.l + t0) * a.g + gg) * N;

    int half = 0;  // the buffer to be read next
    const auto fetch = [&](int64_t hi, int st, int lane) {
        const uint32_t buf = base + half * B::BYTES;
        const int tiles = F32 && cts - 2 * st > 1 ? 2 : 1;
        const int64_t at = hi * cts + B::TILES * st;
        const int whole = tiles * kOperandS<IO, N> * B::E, tok = tiles * kOperandN<IO> * B::E;
        copy_lds(static_cast<const OT *>(a.simg) + at * kOperandS<IO, N>, whole, B::ST, buf + B::S, w, 4,
                 lane);
        copy_lds(static_cast<const OT *>(a.dsimg) + at * kOperandS<IO, N>, whole, B::ST, buf + B::D, w,
                 4, lane);
        copy_lds(static_cast<const OT *>(a.nimg) + at * kOperandN<IO>, tok, B::TOK, buf + B::NV, w, 4,
                 lane);
        copy_lds(static_cast<const OT *>(a.zimg) + at * kOperandN<IO>, tok, B::TOK, buf + B::Z, w, 4,
                 lane);
        copy_lds(static_cast<const OT *>(a.yimg) + at * 1024, tiles * 1024 * B::E, B::TOKY, buf + B::DY, w,
                 4, lane);
        if constexpr (!F32) copy_lds(a.scales + at * kScales, kScales * 4, 1024, buf + B::SC, w, 4, lane);
        if (st == 0) {
            copy_lds(a.rows2 + hi * (kRowsGrad * kDC), kRowsGrad * kDC * 4, kRowsGrad * kDC * 4,
                     base + B::R0, w, 4, lane);
            copy_lds(a.himg + hi * a.hstride + H::R + kBeta * kDC * 4, kDC * 4, 1024, base + B::BETA, w,
                     4, lane);
        }
    };
    const auto fetch_rows = [&](int64_t hi, int lane) {
        const uint32_t buf = base + half * B::BYTES;
        if constexpr (F32) {
            copy_nat<XB>(static_cast<const IO *>(a.k) + kq, a.g * N, N, len, buf + B::K, w, lane);
            copy_nat<XB>(static_cast<const IO *>(a.q) + kq, a.g * N, N, len, buf + B::Q, w, lane);
        } else {
            copy_lds(a.gimg + (ci * a.g + gg) * GroupImg<IO, N>::BYTES, GroupImg<IO, N>::BYTES,
                     GroupImg<IO, N>::BYTES, buf + B::K, w, 4, lane);
        }
        copy_lds(a.himg + hi * a.hstride + H::R, kRows * kDC * 4, kRows * kDC * 4, buf + B::R, w, 4,
                 lane);
        copy_lds(a.rows2 + hi * (kRowsGrad * kDC), kRowsGrad * kDC * 4, kRowsGrad * kDC * 4, buf + B::R2,
                 w, 4, lane);
    };

    f32x4 dQ[NT], dK[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) dQ[x] = dK[x] = zero4();
    // X: N . dY on and above the wave's diagonal tile, dY . N below it, and Xd on
    // it; Y and Yd the same of Z and N
    f32x4 X[4], Y[4], Xd = zero4(), Yd = zero4();
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) X[rt] = Y[rt] = zero4();

    // The next buffer's copies have landed for everyone; the other one is free.  The
    // lane comes out as a value not known to be the same each time: addresses are
    // then computed where they are used, of which there are more than registers.
    const auto turn = [&]() {
        vm_wait<0>();
        lds_barrier();
        const char *buf = lds + half * B::BYTES;
        half ^= 1;
        return buf;
    };
    const auto fresh = [&]() {
        int lane = own;
        asm volatile("" : "+v"(lane));
        return lane;
    };
    const int64_t h0 = ci * a.h + gg * ratio;
    const char *buf = nullptr;
    fetch(h0, 0, own);
    for (int64_t hi = h0; hi < h0 + ratio; ++hi) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) X[rt] = Y[rt] = zero4();
        Xd = Yd = zero4();
        for (int st = 0; st < slices; ++st) {
            buf = turn();
            const int lane = fresh(), g = lane >> 4;
            if (st + 1 < slices)
                fetch(hi, st + 1, lane);
            else
                fetch_rows(hi, lane);
            const OT *S = reinterpret_cast<const OT *>(buf + B::S);
            const OT *D = reinterpret_cast<const OT *>(buf + B::D);
            const OT *NV = reinterpret_cast<const OT *>(buf + B::NV);
            const OT *ZV = reinterpret_cast<const OT *>(buf + B::Z);
            const OT *DY = reinterpret_cast<const OT *>(buf + B::DY);
            // this wave's tokens as second operands: dY; N and Z (`hl`: their two terms);
            // for products with an operand of two terms hi hi and lo hi, then hi lo
            const F dy = cols_nat(DY, w >> 1, NEXTY, w, lane), nhl = cols_nat(NV, w >> 1, NEXT, w, lane);
            F nhh = nhl, zhh = cols_nat(ZV, w >> 1, F32 ? NEXT : 0, w, lane), nl = nhl, zl = zhh;
            if constexpr (!F32) {
                const f16 first = g < 2 ? (f16)1.f : (f16)0.f;
                nhh = cols_nat(NV, w >> 1, 0, w, lane);
                nl = cols_nat(NV, NEXT + (w >> 1), 0, w, lane) * first;
                zl = cols_nat(ZV, NEXT + (w >> 1), 0, w, lane) * first;
            }
            const auto both = [&](const F &x, const F &hh, const F &l) {
                f32x4 t = mma8(x, hh, zero4());
                if constexpr (!F32) t = mma8(x, l, t);
                return t;
            };
            const float *sc = reinterpret_cast<const float *>(buf + B::SC);
            const float *rows = reinterpret_cast<const float *>(lds + B::R0) + 16 * w + (lane & 15);
            const float be = reinterpret_cast<const float *>(lds + B::BETA)[16 * w + (lane & 15)];
            float gq = a.scale * rows[kRead * kDC], gz = -rows[kRead * kDC] * be,
                  gn = rows[kWrite * kDC] * be, ny = 1.f, nz = 1.f;
            float uq = 1.f, uz = 1.f, un = 1.f, uy = 1.f, uzn = 1.f;
            if constexpr (!F32) {
                const Undo q(sc, kScS, kScY), z(sc, kScS, kScZ), n(sc, kScD, kScN), y(sc, kScN, kScY),
                    o(sc, kScN, kScZ);
                gq *= q.a, gz *= z.a, gn *= n.a, ny = y.a, nz = o.a;
                uq = q.b, uz = z.b, un = n.b, uy = y.b, uzn = o.b;
            }
            // to += f (u t); fp32 operands have no u
            const auto add = [&](f32x4 &to, float f, float u, const f32x4 &t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) to[r] = fmaf(f, F32 ? t[r] : u * t[r], to[r]);
            };
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                if (rt <= w) {
                    const F n = cols_nat(NV, rt >> 1, NEXT, rt, lane);
                    add(X[rt], ny, uy, mma8(n, dy, zero4()));
                    add(Y[rt], nz, uzn, both(n, zhh, zl));
                }
                if (rt >= w) {
                    const F d = cols_nat(DY, rt >> 1, NEXTY, rt, lane);
                    const F z = cols_nat(ZV, rt >> 1, NEXT, rt, lane);
                    const f32x4 t = mma8(d, nhl, zero4()), u = both(z, nhh, nl);
                    if (rt == w)
                        add(Xd, ny, uy, t), add(Yd, nz, uzn, u);
                    else
                        add(X[rt], ny, uy, t), add(Y[rt], nz, uzn, u);
                }
                sched_fence();
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const F s = cols_nat(S, x >> 1, XB, x, lane);
                const F d = cols_nat(D, x >> 1, XB, x, lane);
                add(dQ[x], gq, uq, mma8(s, dy, zero4()));
                add(dK[x], gz, uz, both(s, zhh, zl));
                add(dK[x], gn, un, both(d, nhh, nl));
                if (x & 1) sched_fence();
            }
        }
        buf = turn();
        const int lane = fresh(), g = lane >> 4, j16 = lane & 15, m = 16 * w + j16;  // this lane's token
        if (hi + 1 < h0 + ratio) fetch(hi + 1, 0, lane);
        // decays, masks and factors; rows j in front of this token give dq, rows
        // behind it dk, both give (X + X^T) K
        const OT *K = reinterpret_cast<const OT *>(buf + B::K);
        const OT *Q = reinterpret_cast<const OT *>(buf + B::Q);
        const float *rows = reinterpret_cast<const float *>(buf + B::R);
        const float *r2 = reinterpret_cast<const float *>(buf + B::R2);
        // the rows of k and q are the image's times these
        const auto of_k = [&](int rt) { return F32 ? row4(r2, kRk, rt, lane) : row4(rows, kFk, rt, lane); };
        const auto of_q = [&](int rt) {  // and scale
            f32x4 f = F32 ? row4(r2, kRq, rt, lane) : row4(rows, kRawQ, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) f[r] *= a.scale;
            return f;
        };
        const float bm = rows[kBeta * kDC + m];
        f32x4 Dj[4];
        {
            const float hm = r2[kGhi * kDC + m], lm = r2[kGlo * kDC + m], dm = r2[kDoc * kDC + m];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const f32x4 gh = row4(r2, kGhi, rt, lane), gl = row4(r2, kGlo, rt, lane),
                            dj = row4(r2, kDoc, rt, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float G = (gh[r] - hm) + (gl[r] - lm);
                    const float e = exp2_fast(16 * rt + 4 * g + r > m ? G : -G);
                    Dj[rt][r] = dj[r] == dm ? e : 0.f;
                }
            }
        }
        // the terms of the decays' gradient inside the chunk, C_mj for j < m
        {
            // the products' factors; fp32 rows have theirs (1 / norm) taken first, as the
            // products of rows as they come can leave fp32's range
            const float fkm = F32 ? 1.f : rows[kFk * kDC + m];
            const float fqm = F32 ? a.scale : a.scale * rows[kRawQ * kDC + m];
            const float rkm = r2[kRk * kDC + m], rqm = r2[kRq * kDC + m];
            double sum = 0.0;
            double *cells = a.cells + hi * (5 * kDC);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                double col[4] = {0.0, 0.0, 0.0, 0.0};
                if (rt <= w) {
                    f32x4 kk = zero4(), qk = zero4();
                    const float rkj = r2[kRk * kDC + 16 * rt + j16];
#pragma unroll
                    for (int kb = 0; kb < XB; ++kb) {
                        F kj = img_rows(K, rt * XB + kb, lane), qm = img_rows(Q, w * XB + kb, lane),
                          km = img_rows(K, w * XB + kb, lane);
                        if constexpr (F32) kj *= rkj, qm *= rqm, km *= rkm;
                        qk = mma8(kj, qm, qk);
                        kk = mma8(kj, km, kk);
                    }
                    const f32x4 bj = row4(rows, kBeta, rt, lane),
                                fk = F32 ? f32x4{1.f, 1.f, 1.f, 1.f} : of_k(rt);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 16 * rt + 4 * g + r;
                        // the rows' factors first: q k and X are as large as the
                        // squares of the inputs
                        const float cell = bj[r] * Dj[rt][r] *
                                           (X[rt][r] * (fk[r] * (fqm * qk[r])) -
                                            bm * Y[rt][r] * (fk[r] * (fkm * kk[r])));
                        const double v = j < m ? (double)cell : 0.0;
                        sum += v;
                        col[r] = sum16(v);
                    }
                }
                if (j16 == 0)
#pragma unroll
                    for (int r = 0; r < 4; ++r) cells[(1 + w) * kDC + 16 * rt + 4 * g + r] = col[r];
                sched_fence();
            }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (g == 0) cells[m] = sum;
        }
        // the masked products as operands, each token's under a power of two
        const auto put = [&](F (&f)[2], F (&l)[2], const f32x4 (&v)[4]) {
            if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e >> 3][e & 7] = v[e >> 2][e & 3];
                return 1.f;
            } else {
                float mx = 0.f;
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) mx = abs_max(mx, v[rt]);
                const Pow2 p(col_max(mx));
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    const Split s = split8(v[2 * tb], v[2 * tb + 1], p.sc);
                    f[tb] = s.hi, l[tb] = s.lo;
                }
                return p.inv;
            }
        };
        const auto kcols = [&](const OT *img, int tb, int x) {
            if constexpr (F32)
                return nat_cols<XB>(img, 2 * tb, x, lane);
            else
                return img_cols(img, 2 * tb * XB + (x >> 1), (2 * tb + 1) * XB + (x >> 1), x, lane);
        };
        // a block of 32 tokens' share of such a product
        const auto masked = [&](const OT *img, int tb, int x, const F (&f)[2], const F (&l)[2], f32x4 t) {
            const F k = kcols(img, tb, x);
            t = mma8(k, f[tb], t);
            if constexpr (!F32) t = mma8(k, l[tb], t);
            return t;
        };
        f32x4 v[4];
        F f[2], l[2];
        // dQ += K^T (rows j <= m of dY U^T)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 bj = row4(rows, kBeta, rt, lane), fk = of_k(rt);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[rt][r] = rt <= w && 16 * rt + 4 * g + r <= m
                               ? a.scale * bj[r] * fk[r] * Dj[rt][r] * X[rt][r] : 0.f;
        }
        float inv = put(f, l, v);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            f32x4 t = masked(K, 0, x, f, l, zero4());
            if (w >> 1) t = masked(K, 1, x, f, l, t);
#pragma unroll
            for (int r = 0; r < 4; ++r) dQ[x][r] = fmaf(inv, t[r], dQ[x][r]);
            if (x & 1) sched_fence();
        }
        // dK += Q^T (rows i >= m of it)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 fqr = of_q(rt);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float xv = rt == w ? Xd[r] : X[rt][r];
                v[rt][r] = rt >= w && 16 * rt + 4 * g + r >= m ? bm * fqr[r] * Dj[rt][r] * xv : 0.f;
            }
        }
        inv = put(f, l, v);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            f32x4 t = masked(Q, 1, x, f, l, zero4());
            if (!(w >> 1)) t = masked(Q, 0, x, f, l, t);
#pragma unroll
            for (int r = 0; r < 4; ++r) dK[x][r] = fmaf(inv, t[r], dK[x][r]);
            if (x & 1) sched_fence();
        }
        // dK -= K^T (dV U^T and its transpose), this token's beta last: beta's square can
        // leave fp32's range where keys are small or large
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 bj = row4(rows, kBeta, rt, lane), fk = of_k(rt);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * rt + 4 * g + r;
                const float yv = rt == w && j > m ? Yd[r] : Y[rt][r];
                v[rt][r] = j == m ? 0.f : -bj[r] * fk[r] * Dj[rt][r] * yv;
            }
        }
        inv = put(f, l, v) * bm;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            f32x4 t = masked(K, 0, x, f, l, zero4());
            t = masked(K, 1, x, f, l, t);
#pragma unroll
            for (int r = 0; r < 4; ++r) dK[x][r] = fmaf(inv, t[r], dK[x][r]);
            if (x & 1) sched_fence();
        }
    }
    const int lane = own, g = lane >> 4, m = 16 * w + (lane & 15);
    const bool live = m < len;
    const float *rows = reinterpret_cast<const float *>(buf + B::R);
    const float *r2 = reinterpret_cast<const float *>(buf + B::R2);
    const int64_t at = ((bb * a.l + t0 + m) * a.g + gg) * N;
    const float rk = r2[kRk * kDC + m], rq = r2[kRq * kDC + m];
    // k and q as the rule has them, from their images
    const float fk = F32 ? rk : rows[kFk * kDC + m], fqr = F32 ? rq : rows[kRawQ * kDC + m];
    const auto unit = [&](const OT *img, float f, int x) {
        f32x4 v;
        if constexpr (F32) {
            v = nat4<XB>(img, m, 16 * x + 4 * g);
        } else {
            const f16x4 h = *reinterpret_cast<const f16x4 *>(img + img_at(m, 16 * x + 4 * g, XB));
            v = f32x4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= f;
        return v;
    };
    const OT *K = reinterpret_cast<const OT *>(buf + B::K), *Q = reinterpret_cast<const OT *>(buf + B::Q);
    put_rows<NT>(dK, [&](int x) { return unit(K, fk, x); }, static_cast<IO *>(a.dk) + at, rk, a.norm, live,
                 g);
    put_rows<NT>(dQ, [&](int x) { return unit(Q, fqr, x); }, static_cast<IO *>(a.dq) + at, rq, a.norm,
                 live, g);
}

// The gradients of dt and beta, a wave per chunk and head, a lane per token.
template <typename IO> __global__ __launch_bounds__(256) void k_delta_dt(DeltaArgs a) {
    const int lane = threadIdx.x & 63, cts = a.p >> 4;
    const int64_t hi = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (hi >= a.b * a.nc * a.h) return;
    const int64_t hh = hi % a.h, ci = hi / a.h, c = ci % a.nc, bb = ci / a.nc, t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
    // tokens from this one on, and columns in front of it
    double s = 0.0, out = 0.0, zn = 0.0, e = 0.0;
    for (int t = 0; t < cts; ++t) {
        const float *k = a.toks + ((hi * cts + t) * kSums) * kDC + lane;
        s += (double)k[kSumQ * kDC] - (double)k[kSumK * kDC];
        out += (double)k[kSumOut * kDC];
        zn += (double)k[kSumZ * kDC];
        e += (double)a.eend[hi * cts + t];
    }
    const double *cells = a.cells + hi * (5 * kDC) + lane;
    s += cells[0] - ((cells[kDC] + cells[2 * kDC]) + (cells[3 * kDC] + cells[4 * kDC]));
    const double own = out;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_down(s, o), v = __shfl_up(out, o);
        if (lane + o < 64) s += u;
        if (lane >= o) out += v;
    }
    s += (out - own) + e;
    const float *r2 = a.rows2 + hi * (kRowsGrad * kDC);
    const float doc = r2[kDoc * kDC + lane], front = lane ? r2[kDoc * kDC + lane - 1] : 0.f;
    const float step = r2[kStep * kDC + lane];
    const bool in = lane < len;
    // nothing decays in front of a document's first token or of a zero state
    const bool none = doc != front || (t0 + lane == 0 && !a.init);
    const int64_t at = (bb * a.l + t0 + lane) * a.h + hh;
    const double dg = !in || none ? 0.0 : s;
    const float z = in ? to_f32(static_cast<const IO *>(a.dt)[at]) + (a.bias ? a.bias[hh] : 0.f) : 0.f;
    const float open = time_step(z, 0.f, a.softplus, -INFINITY, INFINITY);
    const bool pass = open >= a.lo && open <= a.hi;
    const float slope = !pass ? 0.f : a.softplus ? 1.f / (1.f + expf(-z)) : 1.f;
    double pb = dg * (double)a.A[hh] * (double)slope, pa = dg * (double)step;
    if (in) {
        static_cast<IO *>(a.ddt)[at] = (IO)(float)pb;
        static_cast<IO *>(a.dbeta)[at] = (IO)(float)zn;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) pa += __shfl_xor(pa, o), pb += __shfl_xor(pb, o);
    if (lane == 0) a.part[2 * hi] = pa, a.part[2 * hi + 1] = pb;
}

// dA and ddt_bias: the chunks' sums, in order by 64 strips.
__global__ __launch_bounds__(64) void k_delta_sum(DeltaArgs a) {
    const int64_t hh = blockIdx.x, n = a.b * a.nc;
    double pa = 0.0, pb = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 64) {
        pa += a.part[2 * (i * a.h + hh)];
        pb += a.part[2 * (i * a.h + hh) + 1];
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) pa += __shfl_xor(pa, o), pb += __shfl_xor(pb, o);
    if (threadIdx.x == 0) {
        a.dA[hh] = (float)pa;
        if (a.dbias) a.dbias[hh] = (float)pb;
    }
}

template <typename IO, int N> hipError_t bwd_n(const DeltaArgs &a, hipStream_t s) {
    const int nw = a.p >= 64 ? 4 : a.p / 16;
    const int64_t walks = a.b * a.h * (a.p / (16 * nw));
    // fewer columns to a workgroup where the walk would leave compute units idle
    // (4 x 16 heads of 128 columns, 32 columns: 205 us with twice the copies, 225 with 64)
    int rw = nw;
    while (rw > 1 && a.b * a.h * (a.p / (16 * rw)) < device_cus()) rw >>= 1;
    const int one = RevBuf<IO, N>::bytes(16 * rw);
    const bool two = 2 * one <= kLdsMost;
    hipError_t e = launch(&k_delta_mid<IO, N>, walks * a.nc, 64 * nw,
                          FwdBuf<IO, N, true>::bytes(16 * nw), a, s);
    if (e == hipSuccess)
        e = launch(two ? &k_delta_rev<IO, N, 2> : &k_delta_rev<IO, N, 1>,
                   a.b * a.h * (a.p / (16 * rw)), 64 * rw,
                   two ? 2 * one : one, a, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_delta_grad<IO, N>), dim3((unsigned)(a.b * a.nc * a.g)), dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_delta_dt<IO>, dim3((unsigned)((a.b * a.nc * a.h + 3) / 4)), dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_delta_sum, dim3((unsigned)a.h), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t delta_backward(const DeltaArgs &a, int io, int n, hipStream_t s) {
    if (io == SSD_BF16)
        return n == 32 ? bwd_n<bf16, 32>(a, s) : n == 64 ? bwd_n<bf16, 64>(a, s) : bwd_n<bf16, 128>(a, s);
    return n == 32 ? bwd_n<float, 32>(a, s) : n == 64 ? bwd_n<float, 64>(a, s) : bwd_n<float, 128>(a, s);
}

}  // namespace ssd
