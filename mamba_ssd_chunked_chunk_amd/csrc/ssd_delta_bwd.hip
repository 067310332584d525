// The gated delta rule's gradient (formulas in ssd_delta.hpp), after the forward
// kernels have left the states in front of the chunks, N and dY . Y:
//
// k_delta_rev, chunk after chunk from the end: the adjoint state of 16 value
// columns in a wave's registers, as in the forward pass; leaves Z, dV, the
// adjoint state behind every chunk, and per token dV . V and per chunk <S', dS>,
// from which the decays' gradient follows without q, k or any further product.
//
// k_delta_grad, all chunks in parallel: dq and dk, which contract over the value
// columns.  A wave owns 16 tokens, all keys of them in registers, transposed
// ([key][token]), so that the masked products dY U^T and Z N^T are the next
// product's operands as they stand; the heads that share q and k are walked in
// order by one workgroup.  Its operands are the io type's (bf16, or fp32 on the
// fp32 matrix instructions): nothing of it enters the recurrence.
#include "ssd_delta.hpp"

#include <math.h>

#include "../../include/ssd.h"

namespace ssd {

namespace {

constexpr int kLdsMost = 160 * 1024;

template <typename IO, int N> struct RevBuf {
    typedef GroupImg<IO, N> G;
    typedef HeadImg<IO, true> H;
    static constexpr int K = 0, Q = G::Q, HEAD = H::BYTES - H::R;  // from the row arrays on
    static constexpr int R = G::BYTES, P = R + H::P - H::R, M = R + H::M - H::R, V = R + HEAD;
    static __host__ __device__ int bytes(int cols) { return V + 2 * kDC * cols * (int)sizeof(IO); }
};

// Where a chunk's operands of one head and `cols` columns are; back() moves to
// the chunk in front.
template <typename IO, int N> struct RevSrc {
    typedef RevBuf<IO, N> B;
    const char *grp, *head, *v, *dy;
    int64_t sg, sh, sv;
    uint32_t pitch;
    int rb, len;
    __device__ RevSrc(const DeltaArgs &a, int64_t bb, int64_t hh, int col0, int cols) {
        const int64_t ci = bb * a.nc + a.nc - 1, t0 = (a.nc - 1) * kDC;
        grp = uni(a.gimg + (ci * a.g + hh / (a.h / a.g)) * B::G::BYTES);
        head = uni(a.himg + (ci * a.h + hh) * B::H::BYTES + B::H::R);
        const int64_t at = (((bb * a.l + t0) * a.h + hh) * a.p + col0) * (int64_t)sizeof(IO);
        v = uni(static_cast<const char *>(a.v) + at);
        dy = uni(static_cast<const char *>(a.dy) + at);
        pitch = (uint32_t)(a.h * a.p * sizeof(IO));
        sg = a.g * B::G::BYTES, sh = a.h * B::H::BYTES, sv = (int64_t)kDC * pitch;
        rb = cols * (int)sizeof(IO), len = uni((int)(a.l - t0));
    }
    __device__ void back() { grp -= sg, head -= sh, v -= sv, dy -= sv, len = kDC; }
    __device__ void copy(uint32_t buf, int wave, int nw, int lane) const {
        copy_image<B::G::BYTES>(grp, buf, wave, nw, lane);
        copy_image<B::HEAD>(head, buf + B::R, wave, nw, lane);
        copy_rows(v, pitch, rb, len, buf + B::V, wave, nw, lane);
        copy_rows(dy, pitch, rb, len, buf + B::V + kDC * rb, wave, nw, lane);
    }
};

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

// Sum over a wave's 16 columns of a state in memory times one in accumulators.
template <int NT>
__device__ __forceinline__ float state_dot(const float *st, int p, const f32x4 (&d)[NT], int lane) {
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) s = fmaf(st[(16 * x + 4 * (lane >> 4) + r) * p], d[x][r], s);
    s = sum16(s);
    s += __shfl_xor(s, 16);
    return s + __shfl_xor(s, 32);
}

// The same of an inverse, which is kept transposed.
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

template <typename IO, int N, int NB>
__global__ __launch_bounds__(256, 2) void k_delta_rev(DeltaArgs a) {
    typedef RevBuf<IO, N> B;
    typedef typename Frag8<IO>::type F;
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
    for (int64_t c = a.nc - 1; c >= 0; --c) {
        const char *buf = lds + (NB == 2 ? (c & 1) * bufbytes : 0);
        // the copies of this chunk are older than the last chunk's stores
        if (c == a.nc - 1 || NB == 1)
            vm_wait<0>();
        else
            vm_wait<16 + (F32 ? 4 : 2) + 8 + 1 + (F32 ? NT : NT / 2)>();
        lds_barrier();
        const int64_t hi = (bb * a.nc + c) * a.h + hh, t0 = c * kDC;
        const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
        if (NB == 2 && c > 0) {
            src.back();
            src.copy(base + ((c - 1) & 1) * bufbytes, wave, nw, lane);
        }
        const f16 *K = reinterpret_cast<const f16 *>(buf + B::K);
        const f16 *Q = reinterpret_cast<const f16 *>(buf + B::Q);
        const f16 *M = reinterpret_cast<const f16 *>(buf + B::M);
        const f16 *P = reinterpret_cast<const f16 *>(buf + B::P);
        const float *rows = reinterpret_cast<const float *>(buf + B::R);
        const IO *V = reinterpret_cast<const IO *>(buf + B::V);
        const IO *dY = V + kDC * cols;

        // the adjoint state behind the chunk: split, and kept for k_delta_grad
        float mx = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) mx = abs_max(mx, dS[x]);
        const Pow2 ps(col_max(mx));
        Split sf[XB];
        F *ds = reinterpret_cast<F *>(static_cast<IO *>(a.dsimg) + (hi * cts + ct) * (XB * 512)) + lane;
#pragma unroll
        for (int kb = 0; kb < XB; ++kb) {
            sf[kb] = split8(dS[2 * kb], dS[2 * kb + 1], ps.sc);
            F f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (IO)dS[2 * kb + (e >> 2)][e & 3];
            ds[64 * kb] = f;
        }
        // dY with scale fq, and with e^G too, under one power of two
        f32x4 E[4], G[4];
        mx = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 d = lds_tile(dY, cols, rt, 16 * wave, lane);
            const f32x4 f = row4(rows, kFq, rt, lane), fr = row4(rows, kReadQ, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) E[rt][r] = d[r] * f[r], G[rt][r] = d[r] * fr[r];
            mx = abs_max(mx, E[rt]);
        }
        const Pow2 pe(col_max(mx));
        Split ef[2], gf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            ef[tb] = split8(E[2 * tb], E[2 * tb + 1], pe.sc);
            gf[tb] = split8(G[2 * tb], G[2 * tb + 1], pe.sc);
        }
        // dU = tril(Q K^T)^T dY + e^{G_C - G} K dS
        f32x4 U[4];
        mx = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 x = tri_t(P, rt, ef, lane);
            f32x4 t = zero4();
#pragma unroll
            for (int kb = 0; kb < XB; ++kb) {
                const f16x8 k = img_rows(K, rt * XB + kb, lane);
                t = mma16(k, sf[kb].hi, t);
                t = mma16(k, sf[kb].lo, t);
                if constexpr (F32) t = mma16(img_rows(K + IMG, rt * XB + kb, lane), sf[kb].hi, t);
            }
            const f32x4 fk = row4(rows, kFk, rt, lane), wk = row4(rows, kWriteK, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                U[rt][r] = fmaf(fk[r] * pe.inv, x[r], wk[r] * ps.inv * t[r]);
            mx = abs_max(mx, U[rt]);
        }
        // Z, dV = beta Z, and their rows' products
        const Pow2 pu(col_max(mx));
        Split uf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) uf[tb] = split8(U[2 * tb], U[2 * tb + 1], pu.sc);
        f32x4 Z[4], W[4];
        mx = 0.f;
        const Rsrc rv = make_rsrc(static_cast<IO *>(a.dv) + ((bb * a.l + t0) * a.h + hh) * a.p + col,
                                  (int64_t)(len - 1) * pitch + 16 * sizeof(IO));
        float *dvv = a.dvv + (hi * cts + ct) * kDC;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 t = inv_t(M, rt, uf, lane);
            const f32x4 be = row4(rows, kBeta, rt, lane), rk = row4(rows, kReadK, rt, lane);
            f32x4 d = lds_tile(V, cols, rt, 16 * wave, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                Z[rt][r] = t[r] * pu.inv;
                const float v = be[r] * Z[rt][r];
                W[rt][r] = rk[r] * v;
                buf_put(rv, (16 * rt + 4 * g + r) * pitch + j16 * sizeof(IO), v, IO{});
                d[r] = sum16(d[r] * v);
            }
            mx = abs_max(mx, W[rt]);
            if (j16 == 0) *reinterpret_cast<f32x4 *>(dvv + 16 * rt + 4 * g) = d;
        }
        F *dz = reinterpret_cast<F *>(static_cast<IO *>(a.zimg) + (hi * cts + ct) * (2 * 512)) + lane;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            F f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (IO)Z[2 * tb + (e >> 2)][e & 3];
            dz[64 * tb] = f;
        }
        // dbeta's products Z . N
        {
            const int64_t at = (hi * cts + ct) * (2 * 512) + 8 * lane;
            float *o = a.dzn + (hi * cts + ct) * kDC;
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const F f = *reinterpret_cast<const F *>(static_cast<const IO *>(a.nimg) + at + 512 * tb);
                F low = f;
                if constexpr (!F32)
                    low = *reinterpret_cast<const F *>(static_cast<const IO *>(a.nlow) + at + 512 * tb);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f32x4 d;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int e = 4 * i + r;
                        d[r] = sum16(Z[2 * tb + i][r] * (F32 ? (float)f[e] : (float)f[e] + (float)low[e]));
                    }
                    if (j16 == 0) *reinterpret_cast<f32x4 *>(o + 16 * (2 * tb + i) + 4 * g) = d;
                }
            }
        }
        // <S', dS> of these columns
        const float along = state_dot(a.kept + hi * N * a.p + col + j16, a.p, dS, lane);
        if (lane == 0) a.eend[hi * cts + ct] = along;
        // dS <- e^{G_C} dS + Q^T (scale e^G dY) - K^T (e^G dV)
        const Pow2 pw(col_max(mx));
        Split wf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) wf[tb] = split8(W[2 * tb], W[2 * tb + 1], pw.sc);
        const float carry = rows[kCarry * kDC];
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
    if (a.init) {
        const int64_t bh = bb * a.h + hh;
        const float along = state_dot(a.init + bh * N * a.p + col + j16, a.p, dS, lane);
        if (lane == 0) a.eend[(a.b * a.nc * a.h + bh) * cts + ct] = along;
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
typedef Frag8<bf16>::type bf16x8;
typedef Frag8<float>::type f32x8;
__device__ __forceinline__ f32x4 mma8(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
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

// A token's gradient through the normalisation (the rows as they were are the
// image's, r is 1 / norm), and out: four keys per lane and tile.
template <int NT, typename IO>
__device__ __forceinline__ void put_rows(f32x4 (&d)[NT], const IO *img, IO *out, float r, int norm,
                                         bool live, int m, int g) {
    if (norm) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const f32x4 v = nat4<NT / 2>(img, m, 16 * x + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fmaf(d[x][i], v[i] * r, s);
        }
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const f32x4 v = nat4<NT / 2>(img, m, 16 * x + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[x][i] = r * fmaf(-s, v[i] * r, d[x][i]);
        }
    }
    if (live)
#pragma unroll
        for (int x = 0; x < NT; ++x) st4<IO>(out + 16 * x + 4 * g, d[x]);
}

// One stage of k_delta_grad in LDS: 32 value columns of a head (states in front
// and adjoint states behind as [column][key] images, N and Z as [column][token],
// rows of dY), or its group's rows of k and q with the head's row arrays.
template <typename IO, int N> struct GradBuf {
    static constexpr int E = (int)sizeof(IO);
    static constexpr int S = 0, D = S + N * 32 * E, NV = D + N * 32 * E, Z = NV + kDC * 32 * E;
    static constexpr int DY = Z + kDC * 32 * E, END1 = DY + kDC * 32 * E;
    static constexpr int K = 0, Q = K + kDC * N * E, R = Q + kDC * N * E;
    static constexpr int R2 = R + kRows * kDC * 4, END2 = R2 + kRowsGrad * kDC * 4;
    static constexpr int BYTES = END1 > END2 ? END1 : END2;
};

template <typename IO, int N>
__global__ __launch_bounds__(256, 2) void k_delta_grad(DeltaArgs a) {
    typedef typename Frag8<IO>::type F;
    typedef GradBuf<IO, N> B;
    typedef HeadImg<IO, true> H;
    constexpr int XB = N / 32, NT = N / 16;
    __shared__ __align__(1024) char lds[2 * B::BYTES];

    const int lane = threadIdx.x & 63, w = wave_id(), g = lane >> 4, j16 = lane & 15;
    const int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int64_t gg = item % a.g, ci = item / a.g, c = ci % a.nc, bb = ci / a.nc;
    const int ratio = (int)(a.h / a.g);
    const int64_t t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
    const int cts = a.p >> 4, m = 16 * w + j16;  // this lane's token
    const bool live = m < len;
    const uint32_t base = lds_address(lds);
    const int slices = (a.p + 31) >> 5, stages = slices + 1;
    const int64_t kq = ((bb * a.l + t0) * a.g + gg) * N;

    const auto fetch = [&](int q) {
        const uint32_t buf = base + (q & 1) * B::BYTES;
        const int64_t hh = gg * ratio + q / stages, hi = ci * a.h + hh;
        const int st = q % stages;
        if (st < slices) {
            const int tiles = cts - 2 * st < 2 ? 1 : 2;
            const int64_t at = hi * cts + 2 * st;
            copy_lds(static_cast<const IO *>(a.simg) + at * (XB * 512), tiles * XB * 512 * B::E,
                      N * 32 * B::E, buf + B::S, w, 4, lane);
            copy_lds(static_cast<const IO *>(a.dsimg) + at * (XB * 512), tiles * XB * 512 * B::E,
                      N * 32 * B::E, buf + B::D, w, 4, lane);
            copy_lds(static_cast<const IO *>(a.nimg) + at * 1024, tiles * 1024 * B::E, kDC * 32 * B::E,
                      buf + B::NV, w, 4, lane);
            copy_lds(static_cast<const IO *>(a.zimg) + at * 1024, tiles * 1024 * B::E, kDC * 32 * B::E,
                      buf + B::Z, w, 4, lane);
            copy_nat<1>(static_cast<const IO *>(a.dy) + ((bb * a.l + t0) * a.h + hh) * a.p + 32 * st,
                        a.h * a.p, 16 * tiles, len, buf + B::DY, w, lane);
        } else {
            copy_nat<XB>(static_cast<const IO *>(a.k) + kq, a.g * N, N, len,
                         buf + B::K, w, lane);
            copy_nat<XB>(static_cast<const IO *>(a.q) + kq, a.g * N, N, len,
                         buf + B::Q, w, lane);
            copy_image<kRows * kDC * 4>(uni(a.himg + hi * H::BYTES + H::R), buf + B::R, w, 4, lane);
            copy_lds(a.rows2 + hi * (kRowsGrad * kDC), kRowsGrad * kDC * 4, kRowsGrad * kDC * 4,
                      buf + B::R2, w, 4, lane);
        }
    };

    f32x4 dQ[NT], dK[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) dQ[x] = dK[x] = zero4();
    // X: N . dY on and above the wave's diagonal tile, dY . N below it, and Xd on
    // it; Y and Yd the same of Z and N
    f32x4 X[4], Y[4], Xd = zero4(), Yd = zero4();
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) X[rt] = Y[rt] = zero4();
    float fq = 0.f, fz = 0.f, fn = 0.f;

    fetch(0);
    for (int q = 0; q < ratio * stages; ++q) {
        const int64_t hh = gg * ratio + q / stages, hi = ci * a.h + hh;
        const int st = q % stages;
        const char *buf = lds + (q & 1) * B::BYTES;
        if (st == 0) {
            const float *r2 = a.rows2 + hi * (kRowsGrad * kDC) + m;
            const float be =
                reinterpret_cast<const float *>(a.himg + hi * H::BYTES + H::R)[kBeta * kDC + m];
            fq = a.scale * r2[kRead * kDC], fz = -r2[kRead * kDC] * be, fn = r2[kWrite * kDC] * be;
        }
        vm_wait<0>();
        lds_barrier();
        if (q + 1 < ratio * stages) fetch(q + 1);
        if (st < slices) {
            const IO *S = reinterpret_cast<const IO *>(buf + B::S);
            const IO *D = reinterpret_cast<const IO *>(buf + B::D);
            const IO *NV = reinterpret_cast<const IO *>(buf + B::NV);
            const IO *ZV = reinterpret_cast<const IO *>(buf + B::Z);
            const IO *DY = reinterpret_cast<const IO *>(buf + B::DY);
            const F dy = img_rows(DY, w, lane);
            const F nv = cols_nat(NV, w >> 1, 2, w, lane);
            const F zv = cols_nat(ZV, w >> 1, 2, w, lane);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const F s = cols_nat(S, x >> 1, XB, x, lane);
                const F d = cols_nat(D, x >> 1, XB, x, lane);
                const f32x4 t = mma8(s, dy, zero4()), u = mma8(s, zv, zero4()),
                            v = mma8(d, nv, zero4());
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dQ[x][r] = fmaf(fq, t[r], dQ[x][r]);
                    dK[x][r] = fmaf(fz, u[r], fmaf(fn, v[r], dK[x][r]));
                }
                if (x & 1) sched_fence();
            }
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                if (rt <= w) {
                    const F n = cols_nat(NV, rt >> 1, 2, rt, lane);
                    X[rt] = mma8(n, dy, X[rt]);
                    Y[rt] = mma8(n, zv, Y[rt]);
                }
                if (rt >= w) {
                    const F d = img_rows(DY, rt, lane);
                    const F z = cols_nat(ZV, rt >> 1, 2, rt, lane);
                    if (rt == w) {
                        Xd = mma8(d, nv, Xd);
                        Yd = mma8(z, nv, Yd);
                    } else {
                        X[rt] = mma8(d, nv, X[rt]);
                        Y[rt] = mma8(z, nv, Y[rt]);
                    }
                }
            }
            continue;
        }
        // decays, masks and factors; rows j in front of this token give dq, rows
        // behind it dk, both give (X + X^T) K
        const IO *K = reinterpret_cast<const IO *>(buf + B::K);
        const IO *Q = reinterpret_cast<const IO *>(buf + B::Q);
        const float *bet = reinterpret_cast<const float *>(buf + B::R) + kBeta * kDC;
        const float *r2 = reinterpret_cast<const float *>(buf + B::R2);
        F bq[2], bk[2], bs[2];
        const float hm = r2[kGhi * kDC + m], lm = r2[kGlo * kDC + m], dm = r2[kDoc * kDC + m];
        const float bm = bet[m];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 gh = row4(r2, kGhi, rt, lane), gl = row4(r2, kGlo, rt, lane),
                        dj = row4(r2, kDoc, rt, lane), rk = row4(r2, kRk, rt, lane),
                        rq = row4(r2, kRq, rt, lane), bj = row4(bet, 0, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * rt + 4 * g + r, e = 4 * (rt & 1) + r;
                const float G = (gh[r] - hm) + (gl[r] - lm);
                const float D = dj[r] == dm ? exp2_fast(j > m ? G : -G) : 0.f;
                const float up = rt > w ? 0.f : X[rt][r], lo = rt < w ? 0.f : rt == w ? Xd[r] : X[rt][r];
                const float yu = rt > w ? 0.f : Y[rt][r], yl = rt < w ? 0.f : rt == w ? Yd[r] : Y[rt][r];
                bq[rt >> 1][e] = (IO)(j <= m ? a.scale * bj[r] * rk[r] * D * up : 0.f);
                bk[rt >> 1][e] = (IO)(j >= m ? a.scale * bm * rq[r] * D * lo : 0.f);
                bs[rt >> 1][e] = (IO)(j == m ? 0.f : -bj[r] * bm * rk[r] * D * (j < m ? yu : yl));
            }
            sched_fence();
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) X[rt] = Y[rt] = zero4();
        Xd = Yd = zero4();
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const F k = nat_cols<XB>(K, 2 * tb, x, lane);
                if (tb <= w >> 1) dQ[x] = mma8(k, bq[tb], dQ[x]);
                dK[x] = mma8(k, bs[tb], dK[x]);
                if (tb >= w >> 1) dK[x] = mma8(nat_cols<XB>(Q, 2 * tb, x, lane), bk[tb], dK[x]);
            }
            if (x & 1) sched_fence();
        }
    }
    const char *buf = lds + ((ratio * stages - 1) & 1) * B::BYTES;
    const float *r2 = reinterpret_cast<const float *>(buf + B::R2);
    const int64_t at = ((bb * a.l + t0 + m) * a.g + gg) * N;
    put_rows<NT>(dK, reinterpret_cast<const IO *>(buf + B::K), static_cast<IO *>(a.dk) + at,
                 r2[kRk * kDC + m], a.norm, live, m, g);
    put_rows<NT>(dQ, reinterpret_cast<const IO *>(buf + B::Q), static_cast<IO *>(a.dq) + at,
                 r2[kRq * kDC + m], a.norm, live, m, g);
}

// The gradients of dt and beta, a wave per chunk and head, a lane per token.
template <typename IO> __global__ __launch_bounds__(256) void k_delta_dt(DeltaArgs a) {
    const int lane = threadIdx.x & 63, cts = a.p >> 4;
    const int64_t hi = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (hi >= a.b * a.nc * a.h) return;
    const int64_t hh = hi % a.h, ci = hi / a.h, c = ci % a.nc, bb = ci / a.nc, t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
    double s = 0.0, e = 0.0, zn = 0.0;
    for (int t = 0; t < cts; ++t) {
        const int64_t at = hi * cts + t;
        s += (double)a.doo[at * kDC + lane] - (double)a.dvv[at * kDC + lane];
        zn += (double)a.dzn[at * kDC + lane];
        e += (double)a.eend[at];
    }
    const float *r2 = a.rows2 + hi * (kRowsGrad * kDC);
    const float doc = r2[kDoc * kDC + lane], front = lane ? r2[kDoc * kDC + lane - 1] : 0.f;
    const float step = r2[kStep * kDC + lane];
    // Nothing decays in front of a document's first token or of a zero state, and
    // what is left of a decay below 2^-21 is less than the sums' roundings: the
    // gradient there is zero, and sums do not cross it.
    const bool in = lane < len;
    const bool first = doc != front || (in && a.A[hh] * step < -14.6f);
    const uint64_t cuts = __ballot(first);
    const uint64_t upto = cuts & (~0ull >> (63 - lane)), beyond = lane < 63 ? cuts >> (lane + 1) : 0;
    const int start = upto ? 63 - __clzll((long long)upto) : 0;
    int stop = beyond ? lane + 1 + __ffsll((long long)beyond) - 1 : 64;
    // what follows the token up to the next such one
    if (lane == 63) s += e;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_down(s, o);
        if (lane + o < stop) s += u;
    }
    // In front of the first token of such a run the sum is known: zero, or <S, dS>
    // in front of the chunk.  What it has instead is the roundings', which are
    // spread over the run.
    double known = 0.0;
    if (c || a.init)
        for (int t = 0; t < cts; ++t)
            known += (double)a.eend[(c ? hi - a.h : a.b * a.nc * a.h + bb * a.h + hh) * cts + t];
    stop = stop < len ? stop : len;
    const double off = __shfl(s, start) - (upto ? 0.0 : known);
    if (in) s -= off * (double)(stop - lane) / (double)(stop - start);
    const bool none = first || (t0 + lane == 0 && !a.init);
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
    typedef RevBuf<IO, N> B;
    const int nw = a.p >= 64 ? 4 : a.p / 16, one = B::bytes(16 * nw);
    const dim3 grid((unsigned)(a.b * a.h * (a.p / (16 * nw)))), block(64 * nw);
    const bool two = 2 * one <= kLdsMost;
    auto *k = two ? &k_delta_rev<IO, N, 2> : &k_delta_rev<IO, N, 1>;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, kLdsMost);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, grid, block, two ? 2 * one : one, s, a);
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
