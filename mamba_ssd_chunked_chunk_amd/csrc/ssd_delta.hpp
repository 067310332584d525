// The gated delta rule: what its kernels share (the mathematics, the layout of
// the workspace, operand images).  Per head, with a state S [key_dim, value_dim]:
//
//   P_t = e^{g_t} S_{t-1},  u_t = beta_t (v_t - P_t^T k_t),  S_t = P_t + k_t u_t^T
//   y_t = scale S_t^T q_t,  g_t = A d_t,  d_t = clamp(softplus(dt_t + dt_bias))
//
// In chunks of C = 64 tokens, with G_i the sum of g over the chunk up to token i,
// D_ij = e^{G_i - G_j} (j <= i, same document), S the state in front and
// N_i = v_i - P_i^T k_i (so u = beta N):
//
//   kk = tril(K K^T . D, -1)         T = (I + kk diag(beta))^-1
//   N  = T (V - e^G K S)             U = diag(beta) N
//   Y  = scale (e^G Q S + tril(Q K^T . D) U)
//   S' = e^{G_C} S + K^T (e^{G_C - G} U)
//
// and backwards, with S the state in front, dS that of the state behind:
//
//   dU = scale tril(Q K^T . D)^T dY + e^{G_C - G} K dS
//   Z  = (I + diag(beta) kk)^-T dU,  dV = diag(beta) Z,  dbeta_i = Z_i . N_i
//   dS <- e^{G_C} dS + scale Q^T (e^G dY) - K^T (e^G dV)
//   dQ_i = scale e^{G_i} S dY_i + scale sum_{j<=i} D_ij (dY_i . U_j) k_j
//   dK_j = scale sum_{i>=j} D_ij (dY_i . U_j) q_i - e^{G_j} S dV_j
//          + e^{G_C-G_j} dS U_j - (X + X^T) K,  X_ij = D_ij (dV_i . U_j), j < i
//   dg_t, from the terms that cross token t:
//   C_ij = scale D_ij (q_i . k_j) (dY_i . U_j) - kk_ij (dV_i . U_j),  j <= i
//   dg_t = sum_{i>=t} (scale e^{G_i} dY_i . S^T q_i - e^{G_i} dV_i . S^T k_i)
//          + sum_{i>=t>j} C_ij + sum_{j<t} e^{G_C-G_j} U_j . dS^T k_j + e^{G_C} <S, dS>
//
// A token that starts a document has nothing in front: e^{G} is zero from it
// on, D across it, and e^{G_C - G} in front of the last such token.
//
// Precision.  The products run on fp16 matrix instructions with fp32
// accumulation.  Every operand is an fp32 value times a power of two (per row
// of q, k and tril(Q K^T), per column of a state or of a chunk's rows, one for an
// inverse, so that the largest magnitude fits), written as two fp16 terms hi + lo, 22
// significant bits (fewer below 2^-16 of the largest, of which an element is off by
// 2^-38 at most; the four-wave walk takes bounds for the largest of R, N and the
// update), and multiplied as hi hi + hi lo + lo hi; q and k of bf16 io are exact in
// one.  States, sums, decays and the triangular inverse are fp32, the log decays' sums
// fp64, and so are the sums of C_ij, of which a row's and a column's share all but a few terms.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ssd_device.hpp"

namespace ssd {

constexpr int kDC = 64;       // tokens of a chunk
constexpr int kPieces = 6;    // 16 x 32 pieces of a lower triangular 64 x 64 matrix
constexpr int kRows = 8;      // row arrays of the scans: see RowOf
constexpr int kRowsGrad = 8;  // row arrays of the gradient's last pass

// Per token of a chunk and head, fp32 [array][64].  fk and fq undo the powers
// of two that k and q are stored with (times 1 / norm where the call normalises).
enum RowOf {
    kReadK,   // e^G fk
    kFk,      // fk; for the scans alone what undoes the row's power of two in tril(Q K^T)
    kWriteK,  // e^{G_C - G} fk
    kReadQ,   // scale e^G fq
    kFq,      // scale fq; for the gradient times what undoes that power of two
    kBeta,    // beta
    kCarry,   // see CarryOf
    kRawQ     // fq
};
enum CarryOf {
    kKeep,    // e^{G_C}
    kMostK,   // the largest kReadK
    kMostN,   // a bound of N over the largest |R|: the largest sum of a row of |inverse|
    kMostW,   // the same of beta kWriteK N
    kInvT,    // what undoes the inverses' powers of two
    kInvM
};
enum RowOfGrad {
    kGhi,    // log2 of e^G, as two floats
    kGlo,
    kDoc,    // documents started in the chunk up to the token
    kRead,   // e^G
    kWrite,  // e^{G_C - G}
    kRk,     // 1 / |k| where the call normalises, else 1
    kRq,
    kStep    // d_t
};

// k_delta_grad's operands: with bf16 io two fp16 terms, in two planes, under one power
// of two for 16 value columns of a chunk (of dY, which bf16 holds, one), fp32 otherwise.
template <typename IO> struct GradOp { typedef f16 type; static constexpr int PL = 2; };
template <> struct GradOp<float> { typedef float type; static constexpr int PL = 1; };
enum ScaleOf { kScS, kScD, kScN, kScZ, kScY, kScales = 8 };  // the powers' inverses
// Per token, summed over 16 columns: dY . (scale e^G Q S), dV . (e^G K S),
// U . (e^{G_C - G} K dS) and Z . N.
enum SumOf { kSumQ, kSumK, kSumOut, kSumZ, kSums };

struct DeltaArgs {
    const void *q, *k, *v, *dt, *beta;
    const float *A, *bias, *init;
    const int32_t *seq;
    void *y;
    float *fin, *states;       // written by the forward pass
    const float *kept;         // states of an earlier forward pass
    const void *dy;
    const float *dfin;
    void *dq, *dk, *dv, *ddt, *dbeta;
    float *dA, *dbias, *dinit;
    // workspace
    char *gimg, *himg;  // GroupImg, HeadImg
    float *rows2;
    void *nimg, *zimg, *simg, *dsimg, *yimg;  // operands of k_delta_grad, see GradOp
    float *scales;                            // [chunk, head][16 columns][kScales]
    // e^G K S and tril(Q K^T)^T dY of 16 columns, in accumulator order
    float *g0, *x0;
    float *toks;                              // [chunk, head][16 columns][kSums][64]
    float *eend;
    double *cells, *part;                     // [chunk, head][row sums, 4 column sums][64]
    int64_t hstride;                          // bytes of a HeadImg
    int64_t b, l, h, g, nc;
    int p, softplus, norm;
    float scale, eps, lo, hi;
};

// Operand images.  A matrix M[t][x] (t in tiles of 16, x in blocks of 32) is
// kept as pieces of 64 lanes x 8 elements, piece (t >> 4) * XB + (x >> 5): lane
// (t & 15) + 16 ((x >> 2) & 3) holds, at 4 ((x >> 4) & 1) + (x & 3), element
// (t, x).  So a piece is one operand fragment whose free index is t and whose
// contraction index is x (one 16-byte read per lane, no bank conflicts), four
// consecutive x are contiguous for the transposing read that gives the
// fragment with x free and t contracted, and a copy into LDS is linear.
template <typename T> struct Frag8;
template <> struct Frag8<f16> { typedef f16x8 type; };
template <> struct Frag8<bf16> { typedef __bf16 type __attribute__((ext_vector_type(8))); };
template <> struct Frag8<float> { typedef float type __attribute__((ext_vector_type(8))); };

template <typename T>
__device__ __forceinline__ typename Frag8<T>::type img_rows(const T *img, int piece, int lane) {
    return *reinterpret_cast<const typename Frag8<T>::type *>(img + piece * 512 + lane * 8);
}

// Element offset inside an image of XB blocks a row.
__device__ __forceinline__ int img_at(int t, int x, int XB) {
    return ((t >> 4) * XB + (x >> 5)) * 512 + ((t & 15) + 16 * ((x >> 2) & 3)) * 8 +
           4 * ((x >> 4) & 1) + (x & 3);
}

// Fragment with x free (tile x16) and the 32 contraction indices of pieces p0
// (t = 0..15) and p1 (t = 16..31); x16 & 1 picks the half inside the pieces.
template <typename T>
__device__ __forceinline__ typename Frag8<T>::type img_cols(const T *img, int p0, int p1, int x16,
                                                            int lane) {
    const int g = lane >> 4, j = lane & 15;
    if constexpr (sizeof(T) == 2) {
        const int o = (4 * g + (j >> 2) + 16 * (j & 3)) * 8 + 4 * (x16 & 1);
        const T *a = img + p0 * 512 + o, *b = img + p1 * 512 + o;
        const f16x4 u = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)a));
        const f16x4 w = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)b));
        return __builtin_bit_cast(typename Frag8<T>::type,
                                  f16x8{u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]});
    } else {
        typename Frag8<T>::type r;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = img[(e < 4 ? p0 : p1) * 512 + (4 * g + (e & 3) + 16 * (j >> 2)) * 8 +
                       4 * (x16 & 1) + (j & 3)];
        return r;
    }
}

// Piece of a lower triangular matrix's row tile rt and 32-block kb <= rt / 2.
__device__ __forceinline__ constexpr int tri_piece(int rt, int kb) {
    return rt < 2 ? rt : 2 * rt - 2 + kb;
}

// The same of an inverse, kept transposed (t the column j, x the row i): column
// tile jt and 32-block ib >= jt / 2 of rows.
__device__ __forceinline__ constexpr int tri_piece_t(int jt, int ib) {
    return jt < 2 ? 2 * jt + ib : jt + 2;
}

__device__ __forceinline__ f32x4 mma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Power of two that brings magnitudes up to mx into [2^13, 2^14), and its inverse.
struct Pow2 {
    float sc, inv;
    __device__ explicit Pow2(float mx) {
        const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) & 255;
        int f = 267 - e;
        f = f > 253 ? 253 : f;
        sc = __builtin_bit_cast(float, (uint32_t)f << 23);
        inv = __builtin_bit_cast(float, (uint32_t)(254 - f) << 23);
    }
};

// What divides a row x by sqrt(|x|^2 + eps), for x itself and for sc x, whose sum of
// squares is ss (sc a power of two that brings the row's largest value into [1/2, 1),
// back its inverse): neither |x|^2 nor eps sc^2 need be in fp32's range.
struct UnitRow {
    float of_x, of_scaled;
    __device__ UnitRow(float ss, float sc, float back, float eps) {
        const float e = eps * sc * sc;
        if (ss > 0.f && e < INFINITY) {
            of_scaled = 1.f / sqrtf(ss + e), of_x = of_scaled * sc;
        } else {  // |x|^2 is nothing beside eps; a row of zeros without eps stays that
            of_x = eps > 0.f ? 1.f / sqrtf(eps) : 0.f, of_scaled = ss > 0.f ? of_x * back : 0.f;
        }
    }
};

// hi + lo of two accumulator tiles times sc, as one fragment each (contraction
// over the tiles' rows).
struct Split {
    f16x8 hi, lo;
};
__device__ __forceinline__ Split split8(const f32x4 &a, const f32x4 &b, float sc) {
    Split s;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float x = (i < 4 ? a[i & 3] : b[i & 3]), y = (i < 4 ? a[(i & 3) + 1] : b[(i & 3) + 1]);
        const f16x2 h = __builtin_convertvector(f32x2{x * sc, y * sc}, f16x2);
        s.hi[i] = h[0], s.hi[i + 1] = h[1];
        s.lo[i] = (f16)fmaf(x, sc, -(float)h[0]);
        s.lo[i + 1] = (f16)fmaf(y, sc, -(float)h[1]);
    }
    return s;
}

// One row tile's share of such fragments in LDS ([hi, lo][2 blocks of 32 rows][lane][8]).
__device__ __forceinline__ void put_half(f16 *dst, const f32x4 &v, float sc, int rt, int lane) {
    const f16x2 h0 = __builtin_convertvector(f32x2{v[0] * sc, v[1] * sc}, f16x2);
    const f16x2 h1 = __builtin_convertvector(f32x2{v[2] * sc, v[3] * sc}, f16x2);
    f16 *p = dst + ((rt >> 1) * 64 + lane) * 8 + 4 * (rt & 1);
    *reinterpret_cast<f16x4 *>(p) = f16x4{h0[0], h0[1], h1[0], h1[1]};
    *reinterpret_cast<f16x4 *>(p + 1024) =
        f16x4{(f16)fmaf(v[0], sc, -(float)h0[0]), (f16)fmaf(v[1], sc, -(float)h0[1]),
              (f16)fmaf(v[2], sc, -(float)h1[0]), (f16)fmaf(v[3], sc, -(float)h1[1])};
}

// Largest value over the four lane groups that share a column.  (The swaps'
// results go through scalars: the compiler takes a bit cast of a vector's
// element as one of its first element.)
__device__ __forceinline__ float col_max(float v) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const u2 r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    const uint32_t b = __builtin_bit_cast(
        uint32_t, fmaxf(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1)));
    const u2 s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    return fmaxf(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}
__device__ __forceinline__ float abs_max(float m, const f32x4 &v) {
    return fmaxf(fmaxf(fmaxf(m, fabsf(v[0])), fmaxf(fabsf(v[1]), fabsf(v[2]))), fabsf(v[3]));
}

// Largest value of a wave's 16 columns, in every lane.
template <int CTRL> __device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                                  0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float tile_max(float v) {
    v = dpp_max<0x128>(col_max(v));  // row_ror 8, 4, 2, 1
    v = dpp_max<0x124>(v);
    v = dpp_max<0x122>(v);
    return dpp_max<0x121>(v);
}

// Has the loads of a matrix waited for here, not at their first use: in a loop that
// use would wait for the next chunk's copies too.
template <typename V, int T> __device__ __forceinline__ void landed(V (&v)[T]) {
#pragma unroll
    for (int i = 0; i < T; ++i) asm volatile("" : "+v"(v[i]));
}

// Sum over the 16 lanes of a row of lanes (every lane gets it).
template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                             0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float v) {
    v = dpp_add<0x128>(v);  // row_ror 8, 4, 2, 1
    v = dpp_add<0x124>(v);
    v = dpp_add<0x122>(v);
    return dpp_add<0x121>(v);
}

// lds_dma16 of ssd_device.hpp with the LDS address as a number (uniform, as the
// scalar offset is).
__device__ __forceinline__ void lds_dma16_at(RsrcW r, uint32_t dst, uint32_t voff, uint32_t soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(
                     voff),
                 "s"(r), "s"(dst), "s"(soff)
                 : "memory", "m0");
#else
    (void)r, (void)dst, (void)voff, (void)soff;
#endif
}
__device__ __forceinline__ uint32_t lds_address(char *p) { return (uint32_t)(uintptr_t)(lds_void *)p; }

// What k_delta_prep leaves of a chunk and group (k and q, in PL terms each), and
// of a chunk and head (T, the row arrays, tril(Q K^T) and, for the gradient,
// (I + beta kk)^-1): the scans copy a range of the latter at once.
template <typename IO, int N> struct GroupImg {
    static constexpr int PL = sizeof(IO) / 2, Q = PL * kDC * N * 2, BYTES = 2 * Q;
};
template <bool GRAD> struct HeadImg {
    static constexpr int TRI = kPieces * 1024;
    static constexpr int T = 0, R = 2 * TRI, P = R + kRows * kDC * 4, M = P + 2 * TRI;
    static constexpr int BYTES = M + (GRAD ? 2 * TRI : 0);
};

// Values that are the same in every lane, told to the compiler once (what comes
// out of a 64-bit division is in vector registers).
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char *uni(const void *p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return reinterpret_cast<const char *>(hi << 32 | lo);
}

__device__ __forceinline__ RsrcW uniform_rsrc(const void *base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return RsrcW{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, (uint32_t)kRsrcWord3};
}

// BYTES (a multiple of 1024) of contiguous memory into LDS, a run of them by each
// of `nw` waves.
template <int BYTES>
__device__ __forceinline__ void copy_image(const char *src, uint32_t dst, int wave, int nw, int lane) {
    constexpr int CNT = BYTES >> 10;
    const RsrcW r = uniform_rsrc(src, BYTES);
    for (int i = wave * CNT / nw; i < (wave + 1) * CNT / nw; ++i)
        lds_dma16_at(r, dst + (i << 10), (uint32_t)(lane * 16), (uint32_t)(i << 10));
}

// `bytes` of contiguous memory into LDS by `nw` waves, and zeros up to `all` (a
// multiple of 1024).
__device__ __forceinline__ void copy_lds(const void *src, int bytes, int all, uint32_t dst, int wave,
                                         int nw, int lane) {
    const RsrcW r = make_rsrc_w(src, bytes);
    for (int i = wave; i < all >> 10; i += nw)
        lds_dma16_at(r, dst + (i << 10), (uint32_t)((i << 10) + lane * 16), 0);
}

// 64 rows of `rb` bytes (a power of two from 32 on), `pitch` bytes apart in
// memory, into LDS without gaps.  Rows from `len` on lie beyond the resource and
// come as zeros.
__device__ __forceinline__ void copy_rows(const char *src, uint32_t pitch, int rb, int len,
                                          uint32_t dst, int wave, int nw, int lane) {
    const RsrcW r = uniform_rsrc(src, (uint32_t)(len - 1) * pitch + rb);
    const int sh = 27 - __builtin_clz(rb);  // log2 of the 16-byte parts of a row
    for (int i = wave; i < rb >> 4; i += nw) {
        const int part = i * 64 + lane;
        lds_dma16_at(r, dst + (i << 10), (part >> sh) * pitch + (part & ((1 << sh) - 1)) * 16, 0);
    }
}

// One buffer of LDS: images of k and q, T, tril(Q K^T), the row arrays, then
// the 64 rows of v (and of dy) of the workgroup's columns.
template <typename IO, int N, bool GRAD> struct FwdBuf {
    typedef GroupImg<IO, N> G;
    typedef HeadImg<GRAD> H;
    static constexpr int K = 0, Q = G::Q, HEAD = H::M;
    static constexpr int T = G::BYTES + H::T, R = G::BYTES + H::R, P = G::BYTES + H::P;
    static constexpr int V = G::BYTES + HEAD;
    static __host__ __device__ int bytes(int cols) {
        return V + (GRAD ? 2 : 1) * kDC * cols * (int)sizeof(IO);
    }
};

// Where a chunk's operands of one head and `cols` columns are; next() moves on by
// one chunk.
template <typename IO, int N, bool GRAD> struct FwdSrc {
    typedef FwdBuf<IO, N, GRAD> B;
    const char *grp, *head, *v, *dy;
    int64_t sg, sh, sv;
    uint32_t pitch;
    int rb, left;  // bytes of a row, tokens from here on
    __device__ FwdSrc(const DeltaArgs &a, int64_t bb, int64_t c, int64_t hh, int col0, int cols) {
        const int64_t ci = bb * a.nc + c, t0 = c * kDC;
        grp = uni(a.gimg + (ci * a.g + hh / (a.h / a.g)) * B::G::BYTES);
        head = uni(a.himg + (ci * a.h + hh) * a.hstride);
        const int64_t at = (((bb * a.l + t0) * a.h + hh) * a.p + col0) * (int64_t)sizeof(IO);
        v = uni(static_cast<const char *>(a.v) + at);
        dy = GRAD ? uni(static_cast<const char *>(a.dy) + at) : nullptr;
        pitch = (uint32_t)(a.h * a.p * sizeof(IO));
        sg = a.g * B::G::BYTES, sh = a.h * a.hstride, sv = (int64_t)kDC * pitch;
        rb = cols * (int)sizeof(IO);
        left = uni((int)(a.l - t0));
    }
    __device__ void next() { grp += sg, head += sh, v += sv, dy += sv, left -= kDC; }
    __device__ void copy(uint32_t buf, int wave, int nw, int lane) const {
        copy_image<B::G::BYTES>(grp, buf, wave, nw, lane);
        copy_image<B::HEAD>(head, buf + B::G::BYTES, wave, nw, lane);
        const int len = left < kDC ? left : kDC;
        copy_rows(v, pitch, rb, len, buf + B::V, wave, nw, lane);
        if constexpr (GRAD) copy_rows(dy, pitch, rb, len, buf + B::V + kDC * rb, wave, nw, lane);
    }
};

// Rows 16 rt + 4 g + r of column col0 + (lane & 15) of 64 rows in LDS.
__device__ __forceinline__ f32x4 lds_tile(const bf16 *M, int ld, int rt, int col0, int lane) {
    const f16x4 v = lds_tr4(reinterpret_cast<const f16 *>(M), ld, 16 * rt, col0, lane);
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return f32x4{__builtin_bit_cast(float, w[0] << 16), __builtin_bit_cast(float, w[0] & 0xffff0000u),
                 __builtin_bit_cast(float, w[1] << 16), __builtin_bit_cast(float, w[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 lds_tile(const float *M, int ld, int rt, int col0, int lane) {
    const float *p = M + (16 * rt + 4 * (lane >> 4)) * ld + col0 + (lane & 15);
    return f32x4{p[0], p[ld], p[2 * ld], p[3 * ld]};
}
__device__ __forceinline__ f32x4 row4(const float *rows, int array, int rt, int lane) {
    return *reinterpret_cast<const f32x4 *>(rows + array * kDC + 16 * rt + 4 * (lane >> 4));
}

__device__ __forceinline__ void buf_put(Rsrc r, uint32_t off, float v, bf16) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (bf16)v), r, off, 0, 0);
}
__device__ __forceinline__ void buf_put(Rsrc r, uint32_t off, float v, float) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, 0);
}

int device_cus();
constexpr int kLdsMost = 160 * 1024;

// A kernel with `bytes` of LDS, which may be more than the default's 64 KB.
template <typename K> hipError_t launch(K *k, int64_t items, int threads, int bytes, const DeltaArgs &a,
                                       hipStream_t s) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLdsMost);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3((unsigned)items), dim3(threads), bytes, s, a);
    return hipGetLastError();
}

// Launches (ssd_delta_scan.hip, ssd_delta_bwd.hip).
hipError_t delta_prep(const DeltaArgs &a, int io, int n, bool grad, hipStream_t s);
hipError_t delta_forward(const DeltaArgs &a, int io, int n, hipStream_t s);  // y, states: where given
hipError_t delta_backward(const DeltaArgs &a, int io, int n, hipStream_t s);

}  // namespace ssd
