// The gated delta rule's two forward kernels (formulas in ssd_delta.hpp).
//
// k_delta_prep, all chunks in parallel: everything of a chunk that does not
// depend on the state -- k and q as operand images, the row factors, the
// masked Q K^T and the inverse of the unit triangle.  The inverse is taken in
// 16 x 16 blocks: the four on the diagonal by substitution (a lane per block and
// column), the others by distance from it, T_ij = -T_ii sum_k (kk beta)_ik T_kj,
// on fp32 matrix instructions whose results feed the next product from registers.
// Bound by memory, of which its outputs are most (with keys of 128 and bf16 io 32 KB
// a chunk and group, 26 KB a chunk and head): 65536 tokens of 64 heads, eight to a
// group, 456 us for 2.3 GB; 8 x 2048 tokens of 24 heads with a group each 115 us
// for 0.57 GB; a large copy would take 472 and 117.
//
// k_delta_fwd, chunk after chunk: a wave owns 16 value columns of one head's
// state in registers (an accumulator tile per 16 keys).  Columns do not meet
// anywhere in the recurrence, and an accumulator tile is the operand of the
// next product as it stands, so a wave passes from K S to N to the new state
// without LDS or another wave; LDS holds only what all columns share (the
// images of the next chunk arrive in the other buffer meanwhile).  Bound by
// memory where there are columns enough (8 x 2048 tokens of 24 heads of 128 x 64,
// states kept, 160 us for 0.67 GB), by the chain of one wave, 1200 instructions a
// chunk, where there are fewer: 16 x 1000 tokens of 16 heads of 128 x 128 106 us,
// 0.37 GB.
#include "ssd_delta.hpp"

#include <math.h>

#include "../../include/ssd.h"

namespace ssd {

namespace {

// ------------------------------------------------------------------ prep ---
// Keeps a wave's own LDS stores and loads in program order (the hardware does;
// no barrier is needed as no other wave reads them).
__device__ __forceinline__ void wave_fence() { asm volatile("" ::: "memory"); }

constexpr int kDP = 20;  // pitch of the 16 x 16 blocks in LDS: 16-byte rows, spread over the banks

struct alignas(16) PrepLds {
    float A[4][16 * kDP], X[4][16 * kDP];  // the triangle's diagonal blocks, and their inverses
    float fac[2][kDC], rn[2][kDC];         // row factors of k and q
    float ghi[kDC], glo[kDC], doc[kDC], bet[kDC];
};

// A 16-row tile of k or q as it is in memory, a fragment (contraction over x in
// the order of memory, lane group g the eight from 8 g on) per 32 columns.
template <typename IO, int N> struct RawTile { u32x4 e[N / 32][sizeof(IO) / 2]; };

template <typename IO, int N>
__device__ __forceinline__ void fetch_tile(RawTile<IO, N> &t, const IO *src, int64_t pitch, int rt,
                                           int len, int lane) {
    const int row = 16 * rt + (lane & 15);
    const IO *p = src + row * pitch + 8 * (lane >> 4);
#pragma unroll
    for (int kb = 0; kb < N / 32; ++kb)
#pragma unroll
        for (int i = 0; i < (int)sizeof(IO) / 2; ++i) {
            t.e[kb][i] = u32x4{0, 0, 0, 0};
            if (row < len)
                t.e[kb][i] = *reinterpret_cast<const u32x4 *>(p + 32 * kb + i * (16 / sizeof(IO)));
        }
}
template <int N>
__device__ __forceinline__ void widen(const RawTile<bf16, N> &t, float (&v)[N / 32][8]) {
#pragma unroll
    for (int kb = 0; kb < N / 32; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = t.e[kb][0][i];
            v[kb][2 * i] = __builtin_bit_cast(float, w << 16);
            v[kb][2 * i + 1] = __builtin_bit_cast(float, w & 0xffff0000u);
        }
}
template <int N>
__device__ __forceinline__ void widen(const RawTile<float, N> &t, float (&v)[N / 32][8]) {
#pragma unroll
    for (int kb = 0; kb < N / 32; ++kb)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = t.e[kb][i >> 2][i & 3];
            v[kb][i] = __builtin_bit_cast(float, w);
        }
}

// Brings each row's largest value into [1/2, 1) by a power of two, leaves the
// row's factors in LDS and, if asked, the fragments in the image.
template <typename IO, int N>
__device__ __forceinline__ void use_tile(const DeltaArgs &a, const RawTile<IO, N> &raw, int rt,
                                         float *fac, float *rn, f16 *img, f16x8 (&hi)[N / 32],
                                         f16x8 (&lo)[N / 32], int lane) {
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int XB = N / 32, IMG = kDC * N;
    const int g = lane >> 4, row = 16 * rt + (lane & 15);
    float v[XB][8];
    widen<N>(raw, v);
    float mx = 0.f, ss = 0.f;
#pragma unroll
    for (int kb = 0; kb < XB; ++kb)
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[kb][e]));
    mx = col_max(mx);
    const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) & 255;
    const int f = mx == 0.f ? 127 : 253 - e < 1 ? 1 : 253 - e;
    const float sc = __builtin_bit_cast(float, (uint32_t)f << 23);
    const float back = __builtin_bit_cast(float, (uint32_t)(254 - f) << 23);
#pragma unroll
    for (int kb = 0; kb < XB; ++kb) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[kb][i] *= sc;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const f16x2 h = __builtin_convertvector(f32x2{v[kb][i], v[kb][i + 1]}, f16x2);
            hi[kb][i] = h[0], hi[kb][i + 1] = h[1];
            if constexpr (F32) {
                lo[kb][i] = (f16)(v[kb][i] - (float)h[0]);
                lo[kb][i + 1] = (f16)(v[kb][i + 1] - (float)h[1]);
            }
        }
    }
    // a row of zeros (one behind the last token too) takes no part in bounds of rows
    float factor = mx == 0.f ? 0.f : back, norm = 1.f;
    if (a.norm) {
#pragma unroll
        for (int kb = 0; kb < XB; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[kb][i], v[kb][i], ss);
        ss += __shfl_xor(ss, 16);
        ss += __shfl_xor(ss, 32);
        const UnitRow u(ss, sc, back, a.eps);
        factor = u.of_scaled, norm = u.of_x;
    }
    if (g == 0) fac[row] = factor, rn[row] = norm;
    if (img) {
        // x = 8 g .. 8 g + 7 are two groups of four of the image's order
        f16 *dst = img + (rt * XB * 64 + (lane & 15) + 16 * ((2 * g) & 3)) * 8 + 4 * (g >> 1);
#pragma unroll
        for (int kb = 0; kb < XB; ++kb) {
            const u32x4 w = __builtin_bit_cast(u32x4, hi[kb]);
            *reinterpret_cast<u32x2 *>(dst + kb * 512) = u32x2{w[0], w[1]};
            *reinterpret_cast<u32x2 *>(dst + kb * 512 + 128) = u32x2{w[2], w[3]};
            if constexpr (F32) {
                const u32x4 z = __builtin_bit_cast(u32x4, lo[kb]);
                *reinterpret_cast<u32x2 *>(dst + IMG + kb * 512) = u32x2{z[0], z[1]};
                *reinterpret_cast<u32x2 *>(dst + IMG + kb * 512 + 128) = u32x2{z[2], z[3]};
            }
        }
    }
}

__device__ __forceinline__ constexpr int tri_tile(int i, int j) { return i * (i + 1) / 2 + j; }

// exp2 of a double, by its value in two floats.
__device__ __forceinline__ float exp2_d(double x) {
    const float h = (float)x, e = exp2f(h);
    return fmaf(e, (float)(x - (double)h) * 0.69314718f, e);
}

// A wave takes one chunk and `hs` heads of one group, without a barrier: the
// group's K K^T and Q K^T stay in its registers, transposed (lane: token i = lane
// & 15 of a tile, four consecutive j), which is the form of the triangle's rows
// both as an operand of the inverse's products and in the image.
template <typename IO, int N, bool GRAD>
__global__ __launch_bounds__(256, 2) void k_delta_prep(DeltaArgs a, int hs) {
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int XB = N / 32;
    constexpr int NT = GRAD ? 2 : 1;          // inverses: T, and (I + beta kk)^-1
    __shared__ PrepLds all[4];
    const int lane = threadIdx.x & 63, wave = wave_id(), g = lane >> 4, j16 = lane & 15;
    PrepLds &L = all[wave];
    const int ratio = (int)(a.h / a.g), parts = ratio / hs;
    int64_t item = xcd_item(blockIdx.x, gridDim.x) * 4 + wave;
    if (item >= a.b * a.nc * a.g * parts) return;
    const int part = (int)(item % parts);
    item /= parts;
    const int64_t gg = item % a.g, ci = item / a.g, c = ci % a.nc, bb = ci / a.nc, t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
    const int64_t row0 = ((bb * a.l + t0) * a.g + gg) * N, pitch = a.g * N;

    f32x4 kk[10], qk[10];
    {
        f16x8 kh[4][XB], kl[4][XB], qh[XB], ql[XB];
        typedef GroupImg<IO, N> G;
        f16 *kimg = part ? nullptr : reinterpret_cast<f16 *>(a.gimg + item * G::BYTES);
        f16 *qimg = part ? nullptr : reinterpret_cast<f16 *>(a.gimg + item * G::BYTES + G::Q);
        const IO *ks = static_cast<const IO *>(a.k) + row0, *qs = static_cast<const IO *>(a.q) + row0;
        // all of k in flight at once, and of q what the registers hold beside it
        RawTile<IO, N> kr[4], qr[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) fetch_tile<IO, N>(kr[rt], ks, pitch, rt, len, lane);
#pragma unroll
        for (int rt = 0; rt < (F32 ? 1 : 4); ++rt) fetch_tile<IO, N>(qr[rt], qs, pitch, rt, len, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
            use_tile<IO, N>(a, kr[rt], rt, L.fac[0], L.rn[0], kimg, kh[rt], kl[rt], lane);
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int jt = 0; jt <= it; ++jt) {
                f32x4 t = zero4();
#pragma unroll
                for (int kb = 0; kb < XB; ++kb) {
                    t = mma16(kh[jt][kb], kh[it][kb], t);
                    if constexpr (F32) {
                        t = mma16(kh[jt][kb], kl[it][kb], t);
                        t = mma16(kl[jt][kb], kh[it][kb], t);
                    }
                }
                kk[tri_tile(it, jt)] = t;
            }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            if (F32 && it < 3) fetch_tile<IO, N>(qr[it + 1], qs, pitch, it + 1, len, lane);
            use_tile<IO, N>(a, qr[it], it, L.fac[1], L.rn[1], qimg, qh, ql, lane);
#pragma unroll
            for (int jt = 0; jt <= it; ++jt) {
                f32x4 t = zero4();
#pragma unroll
                for (int kb = 0; kb < XB; ++kb) {
                    t = mma16(kh[jt][kb], qh[kb], t);
                    if constexpr (F32) {
                        t = mma16(kh[jt][kb], ql[kb], t);
                        t = mma16(kl[jt][kb], qh[kb], t);
                    }
                }
                qk[tri_tile(it, jt)] = t;
            }
        }
    }
    for (int64_t hh = gg * ratio + part * hs; hh < gg * ratio + (part + 1) * hs; ++hh) {
        typedef HeadImg<GRAD> H;
        const int64_t hi = ci * a.h + hh;
        char *himg = a.himg + hi * a.hstride;
        float *rows = reinterpret_cast<float *>(himg + H::R);
        // decays: a lane per token
        float load;
        {
            const int64_t at = (bb * a.l + t0 + lane) * a.h + hh;
            const bool in = lane < len;
            double s = 0.0;
            float be = 0.f, step = 0.f;
            if (in) {
                step = time_step(to_f32(static_cast<const IO *>(a.dt)[at]), a.bias ? a.bias[hh] : 0.f,
                                 a.softplus, a.lo, a.hi);
                // below -1e4 e^g is zero all the same, and sums of such steps stay finite
                s = fmax((double)a.A[hh] * (double)step, -1e4) * 1.4426950408889634;
                be = to_f32(static_cast<const IO *>(a.beta)[at]);
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double u = __shfl_up(s, o);
                if (lane >= o) s += u;
            }
            const double end = __shfl(s, 63);
            bool cut = false;
            if (a.seq && in && t0 + lane > 0) {
                const int32_t *q = a.seq + bb * a.l + t0 + lane;
                cut = q[0] != q[-1];
            }
            const uint64_t cuts = __ballot(cut);
            const uint64_t upto = cuts & (~0ull >> (63 - lane));
            const float gh = (float)s, gl = (float)(s - (double)gh), doc = (float)__popcll(upto);
            const float rd = upto ? 0.f : exp2_d(s), wr = upto == cuts ? exp2_d(end - s) : 0.f;
            wave_fence();
            L.ghi[lane] = gh, L.glo[lane] = gl, L.doc[lane] = doc, L.bet[lane] = be;
            const float fk = L.fac[0][lane], fq = L.fac[1][lane];
            float *r = rows + lane;
            r[kReadK * kDC] = rd * fk;
            if constexpr (GRAD) r[kFk * kDC] = fk;
            r[kWriteK * kDC] = wr * fk;
            r[kReadQ * kDC] = a.scale * rd * fq;
            if constexpr (!GRAD) r[kFq * kDC] = a.scale * fq;
            r[kBeta * kDC] = be;
            r[kRawQ * kDC] = fq;
            const float most = tile_max(rd * fabsf(fk));
            load = tile_max(fabsf(be * wr * fk));
            float *carry = rows + kCarry * kDC;
            if (lane == 0) carry[kKeep] = cuts ? 0.f : exp2_d(end), carry[kMostK] = most;
            if constexpr (GRAD) {
                float *e = a.rows2 + hi * (kRowsGrad * kDC) + lane;
                e[kGhi * kDC] = gh;
                e[kGlo * kDC] = gl;
                e[kDoc * kDC] = doc;
                e[kRead * kDC] = rd;
                e[kWrite * kDC] = wr;
                e[kRk * kDC] = L.rn[0][lane];
                e[kRq * kDC] = L.rn[1][lane];
                e[kStep * kDC] = step;
            }
            wave_fence();
        }
        // decays and masks on both triangles
        f32x4 A[10];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i = 16 * it + j16;
            const float gi = L.ghi[i], li = L.glo[i], di = L.doc[i], fi = L.fac[0][i];
            f32x4 pq[4];
            float mx = 0.f;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                pq[jt] = zero4();
                if (jt > it) continue;
                f32x4 bj = f32x4{1.f, 1.f, 1.f, 1.f};
                if constexpr (!GRAD) bj = row4(L.bet, 0, jt, lane);
                const f32x4 gj = row4(L.ghi, 0, jt, lane), lj = row4(L.glo, 0, jt, lane),
                            dj = row4(L.doc, 0, jt, lane), fj = row4(L.fac[0], 0, jt, lane);
                f32x4 d;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = dj[r] == di && (jt < it || 4 * g + r <= j16);
                    const float e = exp2_fast((gi - gj[r]) + (li - lj[r]));
                    d[r] = in ? e : 0.f;
                    const float k = kk[tri_tile(it, jt)][r] * d[r] * (fi * fj[r]);
                    A[tri_tile(it, jt)][r] = jt < it || 4 * g + r < j16 ? k : 0.f;
                    // the read-out takes N: with the factors that make u of it no element
                    // counts that is multiplied by nothing
                    pq[jt][r] = qk[tri_tile(it, jt)][r] * d[r] * (GRAD ? 1.f : bj[r] * fj[r]);
                }
                mx = abs_max(mx, pq[jt]);
            }
            const Pow2 pp(col_max(mx));
            if (g == 0) rows[(GRAD ? kFq : kFk) * kDC + i] = GRAD ? a.scale * L.fac[1][i] * pp.inv : pp.inv;
            f16 *dst = reinterpret_cast<f16 *>(himg + H::P) + lane * 8;
#pragma unroll
            for (int kb = 0; kb <= it / 2; ++kb) {
                const Split s = split8(pq[2 * kb], pq[2 * kb + 1], pp.sc);
                *reinterpret_cast<f16x8 *>(dst + tri_piece(it, kb) * 512) = s.hi;
                *reinterpret_cast<f16x8 *>(dst + (kPieces + tri_piece(it, kb)) * 512) = s.lo;
            }
            *reinterpret_cast<f32x4 *>(&L.A[it][j16 * kDP + 4 * g]) = A[tri_tile(it, it)];
        }
        f32x4 be[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) be[t] = row4(L.bet, 0, t, lane);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
            // diagonal blocks: block g, column j16
            wave_fence();
            float x[16], bx[16];
            const float *K = L.A[g], *bt = L.bet + 16 * g;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s[2] = {0.f, 0.f};  // two chains
#pragma unroll
                for (int k = 0; k < i; ++k) s[k & 1] = fmaf(K[i * kDP + k], bx[k], s[k & 1]);
                const float v = s[0] + s[1];
                x[i] = (i == j16 ? 1.f : 0.f) - (m == 0 ? v : bt[i] * v);
                bx[i] = m == 0 ? bt[i] * x[i] : x[i];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) L.X[g][i * kDP + j16] = x[i];
            wave_fence();
            // the others by their distance from it
            f32x4 T[10], ti[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                ti[t] = *reinterpret_cast<const f32x4 *>(&L.X[t][j16 * kDP + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) T[tri_tile(t, t)][r] = L.X[t][(4 * g + r) * kDP + j16];
            }
#pragma unroll
            for (int d = 1; d < 4; ++d)
#pragma unroll
                for (int j = 0; j < 4 - d; ++j) {
                    const int i = j + d;
                    f32x4 y = zero4(), o = zero4();
#pragma unroll
                    for (int k = j; k < i; ++k)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float t = T[tri_tile(k, j)][q];
                            y = Mfma<float>::mma(A[tri_tile(i, k)][q], m == 0 ? be[k][q] * t : t, y);
                        }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o = Mfma<float>::mma(ti[i][q], m == 0 ? -y[q] : -be[i][q] * y[q], o);
                    T[tri_tile(i, j)] = o;
                }
            float most = 0.f;
#pragma unroll
            for (int t = 0; t < 10; ++t) most = abs_max(most, T[t]);
            const Pow2 pt(tile_max(most));
            float *carry = rows + kCarry * kDC;
            if (lane == 0) carry[m == 0 ? kInvT : kInvM] = pt.inv;
            if (m == 0) {
                most = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 sum = zero4();
#pragma unroll
                    for (int j = 0; j <= i; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) sum[r] += fabsf(T[tri_tile(i, j)][r]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) most = fmaxf(most, sum16(sum[r]));
                }
                most = col_max(most);
                if (lane == 0) carry[kMostN] = most, carry[kMostW] = most * load;
            }
            f16 *dst = reinterpret_cast<f16 *>(himg + (m ? H::M : H::T)) + lane * 8;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
                for (int ib = jt / 2; ib < 2; ++ib) {
                    const f32x4 up = jt > 2 * ib ? zero4() : T[tri_tile(2 * ib, jt > 2 * ib ? 0 : jt)];
                    const Split s = split8(up, T[tri_tile(2 * ib + 1, jt)], pt.sc);
                    *reinterpret_cast<f16x8 *>(dst + tri_piece_t(jt, ib) * 512) = s.hi;
                    *reinterpret_cast<f16x8 *>(dst + (kPieces + tri_piece_t(jt, ib)) * 512) = s.lo;
                }
        }
    }
}

// --------------------------------------------------------------- forward ---
// A workgroup walks all chunks of a head's columns.
template <typename IO, int N, int NB>
__global__ __launch_bounds__(512) void k_delta_fwd(DeltaArgs a) {
    typedef FwdBuf<IO, N, false> B;
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
    const int col = col0 + 16 * wave;
    const int bufbytes = B::bytes(cols);
    const uint32_t base = lds_address(lds);

    FwdSrc<IO, N, false> src(a, bb, 0, hh, col0, cols);
    src.copy(base, wave, nw, lane);
    f32x4 S[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        S[x] = zero4();
        if (a.init)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[x][r] = a.init[((bb * a.h + hh) * N + 16 * x + 4 * g + r) * a.p + col + j16];
    }
    landed(S);
    for (int64_t c = 0; c < a.nc; ++c) {
        const char *buf = lds + (NB == 2 ? (c & 1) * bufbytes : 0);
        // the copies of this chunk are older than the last chunk's stores
        if (c == 0 || NB == 1)
            vm_wait<0>();
        else
            a.states ? vm_wait<16 + 4 * NT>() : vm_wait<16>();
        lds_barrier();
        if (NB == 2 && c + 1 < a.nc) {
            src.next();
            src.copy(base + ((c + 1) & 1) * bufbytes, wave, nw, lane);
        }
        const f16 *K = reinterpret_cast<const f16 *>(buf + B::K);
        const f16 *Q = reinterpret_cast<const f16 *>(buf + B::Q);
        const f16 *T = reinterpret_cast<const f16 *>(buf + B::T);
        const f16 *P = reinterpret_cast<const f16 *>(buf + B::P);
        const float *rows = reinterpret_cast<const float *>(buf + B::R);
        const IO *V = reinterpret_cast<const IO *>(buf + B::V);
        const int64_t t0 = c * kDC, hi = (bb * a.nc + c) * a.h + hh;
        const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);

        // K S and Q S
        float mx = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) mx = abs_max(mx, S[x]);
        const Pow2 ps(col_max(mx));
        Split sf[XB];
#pragma unroll
        for (int kb = 0; kb < XB; ++kb) {
            sf[kb] = split8(S[2 * kb], S[2 * kb + 1], ps.sc);
        }
        f32x4 R[4], Y[4];
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
            const f32x4 v = lds_tile(V, cols, rt, 16 * wave, lane), f = row4(rows, kReadK, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) R[rt][r] = fmaf(-f[r] * ps.inv, t[r], v[r]);
        }
        // N = T R
        mx = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) mx = abs_max(mx, R[rt]);
        const Pow2 pr(col_max(mx));
        Split rf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) rf[tb] = split8(R[2 * tb], R[2 * tb + 1], pr.sc);
        f32x4 U[4], W[4];  // N, and e^{G_C - G} u
        const float undo = pr.inv * rows[kCarry * kDC + kInvT];
        float mw = 0.f;
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
            const f32x4 be = row4(rows, kBeta, rt, lane), wk = row4(rows, kWriteK, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                U[rt][r] = t[r] * undo;
                W[rt][r] = U[rt][r] * be[r] * wk[r];
            }
            mx = abs_max(mx, U[rt]);
            mw = abs_max(mw, W[rt]);
        }
        const Pow2 pu(col_max(mx)), pw(col_max(mw));
        const float carry = rows[kCarry * kDC + kKeep];
        {
            Split wf[2];
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) wf[tb] = split8(W[2 * tb], W[2 * tb + 1], pw.sc);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                f32x4 t = zero4();
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    const int p0 = 2 * tb * XB + (x >> 1), p1 = p0 + XB;
                    const f16x8 k = img_cols(K, p0, p1, x, lane);
                    t = mma16(k, wf[tb].hi, t);
                    t = mma16(k, wf[tb].lo, t);
                    if constexpr (F32) t = mma16(img_cols(K + IMG, p0, p1, x, lane), wf[tb].hi, t);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) S[x][r] = fmaf(t[r], pw.inv, carry * S[x][r]);
            }
        }
        // Y = scale (e^G Q S + tril(Q K^T) U), the latter's image with what makes u of N
        Split uf[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) uf[tb] = split8(U[2 * tb], U[2 * tb + 1], pu.sc);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            f32x4 t = zero4(), u = zero4();
#pragma unroll
            for (int kb = 0; kb < XB; ++kb) {
                const f16x8 q = img_rows(Q, rt * XB + kb, lane);
                t = mma16(q, sf[kb].hi, t);
                t = mma16(q, sf[kb].lo, t);
                if constexpr (F32) t = mma16(img_rows(Q + IMG, rt * XB + kb, lane), sf[kb].hi, t);
            }
#pragma unroll
            for (int tb = 0; tb <= rt / 2; ++tb) {
                const f16x8 p = img_rows(P, tri_piece(rt, tb), lane);
                u = mma16(p, uf[tb].hi, u);
                u = mma16(p, uf[tb].lo, u);
                u = mma16(img_rows(P + kPieces * 512, tri_piece(rt, tb), lane), uf[tb].hi, u);
            }
            const f32x4 fr = row4(rows, kReadQ, rt, lane), fp = row4(rows, kFq, rt, lane),
                        fi = row4(rows, kFk, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                Y[rt][r] = fmaf(fr[r] * ps.inv, t[r], fp[r] * (fi[r] * (pu.inv * u[r])));
        }
        {
            const uint32_t pitch = (uint32_t)(a.h * a.p * sizeof(IO));
            const Rsrc ry = make_rsrc(static_cast<IO *>(a.y) +
                                          ((bb * a.l + t0) * a.h + hh) * a.p + col,
                                      (int64_t)(len - 1) * pitch + 16 * sizeof(IO));
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    buf_put(ry, (16 * rt + 4 * g + r) * pitch + j16 * sizeof(IO), Y[rt][r], IO{});
        }
        if (a.states) {
            float *st = a.states + hi * N * a.p + col;
            const Rsrc rs = make_rsrc(st, ((int64_t)(N - 1) * a.p + 16) * 4);
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    buf_put(rs, (uint32_t)(((16 * x + 4 * g + r) * a.p + j16) * 4), S[x][r], 0.f);
        }
        if (NB == 1 && c + 1 < a.nc) {
            lds_barrier();  // everyone is done with the buffer
            src.next();
            src.copy(base, wave, nw, lane);
        }
    }
    if (a.fin) {
        float *dst = a.fin + (bb * a.h + hh) * N * a.p + col + j16;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(16 * x + 4 * g + r) * a.p] = S[x][r];
    }
}

// The same walk by four waves to 16 columns, for calls with few of them (the
// chain of chunks is then all there is to wait for, and a wave alone issues one
// instruction in four cycles).  A wave owns a quarter of the keys' rows of the
// state and the rows of one of the four row tiles; what it has of K S and Q S
// goes to the rows' owners, and R, N and e^{G_C - G} u, split, to everyone, through
// LDS, with a barrier after each.  There are three stretches between barriers (the end
// of a chunk and the start of the next one are the same), and every place is written in
// one and read in the one after it, so that no two of them may be the same bytes: a wave
// still reads Q S while another writes the next chunk's K S.  With bf16 io Q S has a
// place of its own (65536 tokens of 64 heads of 128 x 64: 3.03 ms against 3.10 with a
// fourth barrier); with fp32 io it takes that of K S, which a fourth barrier in front of
// its next use allows: LDS then holds two buffers with keys of 64 (8192 tokens of 32
// heads of 64 x 64: 365 against 371 us), and with keys of 128 the barrier is the faster
// one too (447 against 452).  The powers of two that the waves have to share come from
// bounds that they exchange with the values before.  65536 tokens of 64 heads of 128 x
// 64: 2.51 us a chunk; operands read from LDS a chunk ahead saved 1% of it, a wait for
// the next chunk's copies moved to the end of this one cost 3%.
template <typename IO> struct CoopBuf {
    static constexpr bool SHARED = sizeof(IO) == 4;  // Q S in the place of K S
    static constexpr int P = 0, Q = SHARED ? P : P + 12 * 1024, R = Q + 12 * 1024, W = R + 4 * 1024;
    static constexpr int U = W + 4 * 1024;
    static constexpr int M = U + 4 * 1024, BYTES = M + 3 * 4 * 64;
};

// LDS leaves room for one workgroup a unit.  (Told so, the compiler spills nothing with
// fp32 keys of 128, 448 against 492 us; with bf16 it gains nothing by it.)
template <typename IO, int N, int NB>
__global__ __launch_bounds__(256, sizeof(IO) == 4 ? 1 : 2) void k_delta_coop(DeltaArgs a) {
    typedef FwdBuf<IO, N, false> B;
    typedef CoopBuf<IO> X;
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int PL = F32 ? 2 : 1, XB = N / 32, NT = N / 16, IMG = kDC * N;
    constexpr int TPW = NT / 4 > 0 ? NT / 4 : 1;  // key tiles of a wave
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, w = wave_id(), g = lane >> 4, j16 = lane & 15;
    int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int cts = a.p >> 4, col = (int)(item % cts) * 16;
    item /= cts;
    const int64_t hh = item % a.h, bb = item / a.h;
    const int bufbytes = B::bytes(16);
    const uint32_t base = lds_address(lds);
    char *ex = lds + NB * bufbytes;
    f32x4 *part = reinterpret_cast<f32x4 *>(ex + X::P);        // [to wave][3 others][lane]
    f32x4 *qpart = reinterpret_cast<f32x4 *>(ex + X::Q);       // the same of Q S
    f16 *rfr = reinterpret_cast<f16 *>(ex + X::R);              // [hi, lo][32 tokens][lane][8]
    f16 *wfr = reinterpret_cast<f16 *>(ex + X::W);
    f16 *ufr = reinterpret_cast<f16 *>(ex + X::U);
    float *mxs = reinterpret_cast<float *>(ex + X::M);          // [S, V, R][wave][column]
    const bool owner = TPW * w < NT;                            // key_dim 32 has two tiles
    const int x0 = TPW * w, kb = x0 >> 1;
    const uint32_t pitch = (uint32_t)(a.h * a.p * sizeof(IO));

    FwdSrc<IO, N, false> src(a, bb, 0, hh, col, 16);
    src.copy(base, w, 4, lane);
    f32x4 S[TPW];
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
        S[x] = zero4();
        if (a.init && owner)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[x][r] = a.init[((bb * a.h + hh) * N + 16 * (x0 + x) + 4 * g + r) * a.p + col + j16];
    }
    landed(S);
    vm_wait<0>();
    lds_barrier();
    for (int64_t c = 0; c < a.nc; ++c) {
        const char *buf = lds + (NB == 2 ? (c & 1) * bufbytes : 0);
        if (NB == 2 && c + 1 < a.nc) {
            src.next();
            src.copy(base + ((c + 1) & 1) * bufbytes, w, 4, lane);
        }
        const f16 *K = reinterpret_cast<const f16 *>(buf + B::K);
        const f16 *Q = reinterpret_cast<const f16 *>(buf + B::Q);
        const f16 *T = reinterpret_cast<const f16 *>(buf + B::T);
        const f16 *P = reinterpret_cast<const f16 *>(buf + B::P);
        const float *rows = reinterpret_cast<const float *>(buf + B::R);
        const IO *V = reinterpret_cast<const IO *>(buf + B::V);
        const int64_t t0 = c * kDC, hi = (bb * a.nc + c) * a.h + hh;
        const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);

        // all of the chunk's operands into registers
        f16x8 kf[PL][4], qf[PL][4], kc[PL][TPW][2], tf[2][2], pf[2][2];
#pragma unroll
        for (int i = 0; i < PL; ++i)
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                kf[i][rt] = img_rows(K + i * IMG, rt * XB + kb, lane);
                qf[i][rt] = img_rows(Q + i * IMG, rt * XB + kb, lane);
            }
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const int b = tb <= w >> 1 ? tb : 0;  // blocks beyond the diagonal are not used
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                tf[i][tb] = img_cols(T + i * kPieces * 512, tri_piece_t(2 * b, w >> 1),
                                     tri_piece_t(2 * b + 1, w >> 1), w, lane);
                pf[i][tb] = img_rows(P + i * kPieces * 512, tri_piece(w, b), lane);
            }
#pragma unroll
            for (int i = 0; i < PL; ++i)
#pragma unroll
                for (int x = 0; x < TPW; ++x) {
                    const int t = owner ? x0 + x : 0;
                    kc[i][x][tb] = img_cols(K + i * IMG, 2 * tb * XB + (t >> 1),
                                            (2 * tb + 1) * XB + (t >> 1), t, lane);
                }
        }
        const f32x4 v = lds_tile(V, 16, w, 0, lane);
        const f32x4 fr = row4(rows, kReadK, w, lane), fi = row4(rows, kFk, w, lane),
                    wk = row4(rows, kWriteK, w, lane), be = row4(rows, kBeta, w, lane),
                    yr = row4(rows, kReadQ, w, lane), yp = row4(rows, kFq, w, lane);
        const float *head = rows + kCarry * kDC;
        const float carry = head[kKeep], mostf = head[kMostK], mostn = head[kMostN],
                    mostw = head[kMostW], invt = head[kInvT];

        // this wave's part of K S and Q S
        float mx = 0.f;
#pragma unroll
        for (int x = 0; x < TPW; ++x) mx = abs_max(mx, S[x]);
        mx = col_max(mx);
        const Pow2 ps(mx);
        // half a block where a wave has one tile
        const Split sf = TPW == 2 ? split8(S[0], S[TPW - 1], ps.sc)
                                  : split8(x0 & 1 ? zero4() : S[0], x0 & 1 ? S[0] : zero4(), ps.sc);
        const float mv = col_max(abs_max(0.f, v));
        if (g == 0) mxs[w * 16 + j16] = mx, mxs[64 + w * 16 + j16] = mv;
        f32x4 ks[4], qs[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            ks[rt] = mma16(kf[0][rt], sf.hi, zero4());
            qs[rt] = mma16(qf[0][rt], sf.hi, zero4());
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            ks[rt] = mma16(kf[0][rt], sf.lo, ks[rt]);
            qs[rt] = mma16(qf[0][rt], sf.lo, qs[rt]);
            if constexpr (F32) {
                ks[rt] = mma16(kf[PL - 1][rt], sf.hi, ks[rt]);
                qs[rt] = mma16(qf[PL - 1][rt], sf.hi, qs[rt]);
            }
        }
        f32x4 mine = zero4(), myq = zero4();
        if constexpr (X::SHARED) lds_barrier();  // everyone has read the last chunk's Q S
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
#pragma unroll
            for (int r = 0; r < 4; ++r) ks[rt][r] *= ps.inv, qs[rt][r] *= ps.inv;
            if (rt == w)
                mine = ks[rt], myq = qs[rt];
            else
                part[(rt * 3 + (w < rt ? w : w - 1)) * 64 + lane] = ks[rt];
        }
        lds_barrier();
        if (NB == 1 && c + 1 < a.nc) {
            src.next();
            src.copy(base, w, 4, lane);
        }
        // R of this wave's rows
        f32x4 R;
        {
            const f32x4 p0 = part[(w * 3) * 64 + lane], p1 = part[(w * 3 + 1) * 64 + lane],
                        p2 = part[(w * 3 + 2) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                R[r] = fmaf(-fr[r], (p0[r] + p1[r]) + (p2[r] + mine[r]), v[r]);
        }
        // |R| <= max |v| + kReadK sum over the keys of |k| |S|, with |k| < 1 here
        float top = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, mxs[64 + i * 16 + j16]), sum += mxs[i * 16 + j16];
        const Pow2 pr(fmaf(mostf * (16.f * TPW), sum, top));
        const float mr = col_max(abs_max(0.f, R));
        if (g == 0) mxs[128 + w * 16 + j16] = mr;
        put_half(rfr, R, pr.sc, w, lane);
        lds_barrier();
        // N = T R, and e^{G_C - G} u
        f32x4 n = zero4();
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
            if (tb <= w >> 1) {
                const f16x8 rh = img_rows(rfr, tb, lane), rl = img_rows(rfr + 1024, tb, lane);
                n = mma16(tf[0][tb], rh, n);
                n = mma16(tf[0][tb], rl, n);
                n = mma16(tf[1][tb], rh, n);
            }
        f32x4 W;
        const float undo = pr.inv * invt;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            n[r] *= undo;
            W[r] = n[r] * be[r] * wk[r];
        }
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, mxs[128 + i * 16 + j16]);
        const Pow2 pu(mostn * top), pw(mostw * top);
        put_half(wfr, W, pw.sc, w, lane);
        put_half(ufr, n, pu.sc, w, lane);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
            if (rt != w) qpart[(rt * 3 + (w < rt ? w : w - 1)) * 64 + lane] = qs[rt];
        vm_wait<0>();
        lds_barrier();
        // this wave's rows of the state
        f32x4 t[TPW];
#pragma unroll
        for (int x = 0; x < TPW; ++x) t[x] = zero4();
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const f16x8 wh = img_rows(wfr, tb, lane), wl = img_rows(wfr + 1024, tb, lane);
#pragma unroll
            for (int x = 0; x < TPW; ++x) {
                t[x] = mma16(kc[0][x][tb], wh, t[x]);
                t[x] = mma16(kc[0][x][tb], wl, t[x]);
                if constexpr (F32) t[x] = mma16(kc[PL - 1][x][tb], wh, t[x]);
            }
        }
#pragma unroll
        for (int x = 0; x < TPW; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[x][r] = owner ? fmaf(t[x][r], pw.inv, carry * S[x][r]) : 0.f;
        if (a.states && owner) {
            float *st = a.states + hi * N * a.p + col + j16;
#pragma unroll
            for (int x = 0; x < TPW; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) st[(16 * (x0 + x) + 4 * g + r) * a.p] = S[x][r];
        }
        // and of Y
        {
            f32x4 y = zero4();
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
                if (tb <= w >> 1) {
                    const f16x8 uh = img_rows(ufr, tb, lane);
                    y = mma16(pf[0][tb], uh, y);
                    y = mma16(pf[0][tb], img_rows(ufr + 1024, tb, lane), y);
                    y = mma16(pf[1][tb], uh, y);
                }
            const f32x4 p0 = qpart[(w * 3) * 64 + lane], p1 = qpart[(w * 3 + 1) * 64 + lane],
                        p2 = qpart[(w * 3 + 2) * 64 + lane];
            const Rsrc ry = make_rsrc(static_cast<IO *>(a.y) + ((bb * a.l + t0) * a.h + hh) * a.p + col,
                                      (int64_t)(len - 1) * pitch + 16 * sizeof(IO));
#pragma unroll
            for (int r = 0; r < 4; ++r)
                buf_put(ry, (16 * w + 4 * g + r) * pitch + j16 * sizeof(IO),
                        fmaf(yr[r], (p0[r] + p1[r]) + (p2[r] + myq[r]),
                             yp[r] * (fi[r] * (pu.inv * y[r]))), IO{});
        }
    }
    if (a.fin && owner) {
        float *dst = a.fin + (bb * a.h + hh) * N * a.p + col + j16;
#pragma unroll
        for (int x = 0; x < TPW; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(16 * (x0 + x) + 4 * g + r) * a.p] = S[x][r];
    }
}

template <typename IO, int N> hipError_t run_fwd(const DeltaArgs &a, hipStream_t s) {
    // columns of a workgroup: all of a head's where that still gives every
    // compute unit a workgroup (its images are then copied once), else 64
    int nw = a.p / 16;
    if (nw > 4 && a.b * a.h < device_cus()) nw = 4;
    const int one = FwdBuf<IO, N, false>::bytes(16 * nw);
    const int64_t items = a.b * a.h * (a.p / (16 * nw));
    const bool two = 2 * one <= kLdsMost;
    return launch(two ? &k_delta_fwd<IO, N, 2> : &k_delta_fwd<IO, N, 1>, items, 64 * nw,
                  two ? 2 * one : one, a, s);
}

template <typename IO, int N> hipError_t prep_n(const DeltaArgs &a, bool grad, hipStream_t s) {
    // heads of a wave: as many of a group as leave eight waves to a compute unit
    const int64_t groups = a.b * a.nc * a.g, ratio = a.h / a.g;
    int64_t hs = ratio;
    while (hs > 1 && (ratio % hs || groups * (ratio / hs) < 8 * device_cus())) --hs;
    const dim3 grid((unsigned)((groups * (ratio / hs) + 3) / 4)), block(256);
    if (grad)
        hipLaunchKernelGGL((k_delta_prep<IO, N, true>), grid, block, 0, s, a, (int)hs);
    else
        hipLaunchKernelGGL((k_delta_prep<IO, N, false>), grid, block, 0, s, a, (int)hs);
    return hipGetLastError();
}

template <typename IO, int N> hipError_t run_coop(const DeltaArgs &a, hipStream_t s) {
    const int one = FwdBuf<IO, N, false>::bytes(16), ex = CoopBuf<IO>::BYTES;
    const bool two = 2 * one + ex <= kLdsMost;
    return launch(two ? &k_delta_coop<IO, N, 2> : &k_delta_coop<IO, N, 1>, a.b * a.h * (a.p / 16), 256,
                  (two ? 2 : 1) * one + ex, a, s);
}

template <typename IO, int N> hipError_t fwd_n(const DeltaArgs &a, hipStream_t s) {
    // Four waves to 16 columns where each such group can have a compute unit of
    // its own; with more of them the chains hide each other's waits.  4096 tokens,
    // keys of 128, heads of 64 columns, 256 compute units: 128, 256, 320 and 768
    // groups take 197, 221, 399 and 661 us by four waves each, 285, 305, 333 and 427
    // by one (fp32 256, 339, 593, 964 and 404, 492, 538, 680; with other widths of
    // keys and columns the two cross between 256 and 320 groups too).
    return a.b * a.h * (a.p / 16) <= device_cus() ? run_coop<IO, N>(a, s) : run_fwd<IO, N>(a, s);
}

}  // namespace

hipError_t delta_prep(const DeltaArgs &a, int io, int n, bool grad, hipStream_t s) {
    if (io == SSD_BF16)
        return n == 32 ? prep_n<bf16, 32>(a, grad, s)
                       : n == 64 ? prep_n<bf16, 64>(a, grad, s) : prep_n<bf16, 128>(a, grad, s);
    return n == 32 ? prep_n<float, 32>(a, grad, s)
                   : n == 64 ? prep_n<float, 64>(a, grad, s) : prep_n<float, 128>(a, grad, s);
}

hipError_t delta_forward(const DeltaArgs &a, int io, int n, hipStream_t s) {
    if (io == SSD_BF16)
        return n == 32 ? fwd_n<bf16, 32>(a, s) : n == 64 ? fwd_n<bf16, 64>(a, s) : fwd_n<bf16, 128>(a, s);
    return n == 32 ? fwd_n<float, 32>(a, s) : n == 64 ? fwd_n<float, 64>(a, s) : fwd_n<float, 128>(a, s);
}

}  // namespace ssd
