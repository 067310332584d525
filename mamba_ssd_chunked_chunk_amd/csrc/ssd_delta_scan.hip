// The gated delta rule's two forward kernels (formulas in ssd_delta.hpp).
//
// k_delta_prep, all chunks in parallel: everything of a chunk that does not
// depend on the state -- k and q as operand images, the row factors, the
// masked Q K^T and the inverse of the unit triangle.  The inverse is taken in
// 16 x 16 blocks: the four on the diagonal by substitution (a lane per column),
// the others by distance from it, T_ij = -T_ii sum_k (kk beta)_ik T_kj, on fp32
// matrix instructions whose results feed the next product from registers.
//
// k_delta_fwd, chunk after chunk: a wave owns 16 value columns of one head's
// state in registers (an accumulator tile per 16 keys).  Columns do not meet
// anywhere in the recurrence, and an accumulator tile is the operand of the
// next product as it stands, so a wave passes from K S to N to the new state
// without LDS or another wave; LDS holds only what all columns share (the
// images of the next chunk arrive in the other buffer meanwhile).
#include "ssd_delta.hpp"

#include <math.h>

#include "../../include/ssd.h"

namespace ssd {

int device_cus();

namespace {

// ------------------------------------------------------------------ prep ---
constexpr int kTP = kDC + 4;  // pitch of the fp32 triangles in LDS

template <typename IO, int N, bool GRAD>
__global__ __launch_bounds__(256) void k_delta_prep(DeltaArgs a) {
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int PL = F32 ? 2 : 1, XB = N / 32, Q4 = N / 4;
    constexpr int IMG = kDC * N;                   // elements of an image
    constexpr int NT = GRAD ? 2 : 1;               // triangles: T, and (I + beta kk)^-1
    constexpr int PPL = F32 || GRAD ? 2 : 1;       // terms of tril(Q K^T)
    __shared__ __align__(16) f16 kq[2][PL * IMG];  // k, q
    __shared__ __align__(16) float tri[1 + NT][kDC * kTP];  // kk, then its inverses
    __shared__ __align__(16) f16 pst[PPL][kPieces * 512];
    __shared__ float fac[2][kDC], rn[2][kDC], ghi[kDC], glo[kDC], bet[kDC], rd[kDC], wr[kDC];
    __shared__ int doc[kDC];

    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), g = lane >> 4, j16 = lane & 15;
    const int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int64_t hh = item % a.h, ci = item / a.h, c = ci % a.nc, bb = ci / a.nc;
    const int ratio = (int)(a.h / a.g);
    const int64_t gg = hh / ratio, t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);

    // rows of k and q: a quarter row per thread
    {
        const int row = tid >> 2, part = tid & 3;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const IO *src = static_cast<const IO *>(m ? a.q : a.k) +
                            ((bb * a.l + t0 + row) * a.g + gg) * N + part * Q4;
            float v[Q4];
#pragma unroll
            for (int i = 0; i < Q4; i += 4) {
                const f32x4 w = row < len ? ld4<IO>(src + i) : zero4();
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i + e] = w[e];
            }
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < Q4; ++i) mx = fmaxf(mx, fabsf(v[i]));
            mx = fmaxf(mx, __shfl_xor(mx, 1));
            mx = fmaxf(mx, __shfl_xor(mx, 2));
            // a power of two that brings the row's largest value into [1/2, 1)
            const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) & 255;
            const int f = mx == 0.f ? 127 : 253 - e < 1 ? 1 : 253 - e;
            const float sc = __builtin_bit_cast(float, (uint32_t)f << 23);
            const float back = __builtin_bit_cast(float, (uint32_t)(254 - f) << 23);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < Q4; ++i) v[i] *= sc, ss = fmaf(v[i], v[i], ss);
            ss += __shfl_xor(ss, 1);
            ss += __shfl_xor(ss, 2);
            // |row|^2 = ss / sc^2: the norm without leaving fp32's range
            const float unit = ss > 0.f ? 1.f / sqrtf(fmaf(a.eps * sc, sc, ss)) : 0.f;
            if (part == 0) {
                fac[m][row] = a.norm ? unit : back;
                rn[m][row] = a.norm ? unit * sc : 1.f;
            }
#pragma unroll
            for (int i = 0; i < Q4; i += 4) {
                const f16x2 h0 = __builtin_convertvector(f32x2{v[i], v[i + 1]}, f16x2);
                const f16x2 h1 = __builtin_convertvector(f32x2{v[i + 2], v[i + 3]}, f16x2);
                const int at = img_at(row, part * Q4 + i, XB);
                *reinterpret_cast<f16x4 *>(&kq[m][at]) = f16x4{h0[0], h0[1], h1[0], h1[1]};
                if constexpr (F32)
                    *reinterpret_cast<f16x4 *>(&kq[m][IMG + at]) =
                        f16x4{(f16)(v[i] - (float)h0[0]), (f16)(v[i + 1] - (float)h0[1]),
                              (f16)(v[i + 2] - (float)h1[0]), (f16)(v[i + 3] - (float)h1[1])};
            }
        }
    }
    for (int i = tid; i < PPL * kPieces * 64; i += 256)
        reinterpret_cast<u32x4 *>(&pst[0][0])[i] = u32x4{0, 0, 0, 0};
    float step = 0.f;
    if (wave == 0) {  // decays: a lane per token
        const int64_t at = (bb * a.l + t0 + lane) * a.h + hh;
        const bool in = lane < len;
        double s = 0.0;
        float be = 0.f;
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
        ghi[lane] = (float)s;
        glo[lane] = (float)(s - (double)(float)s);
        doc[lane] = __popcll(upto);
        bet[lane] = be;
        rd[lane] = upto ? 0.f : exp2f((float)s);
        wr[lane] = upto == cuts ? exp2f((float)(end - s)) : 0.f;
        if (lane == 0)
            a.rows[((ci * a.h + hh) * kRows + kCarry) * kDC] = cuts ? 0.f : exp2f((float)end);
    }
    __syncthreads();

    if (hh % ratio == 0) {
        f16 *dst[2] = {a.kimg + (ci * a.g + gg) * (PL * IMG), a.qimg + (ci * a.g + gg) * (PL * IMG)};
        for (int i = tid; i < PL * IMG / 8; i += 256)
#pragma unroll
            for (int m = 0; m < 2; ++m)
                reinterpret_cast<u32x4 *>(dst[m])[i] = reinterpret_cast<const u32x4 *>(kq[m])[i];
    }
    if (tid < kDC) {
        float *r = a.rows + (ci * a.h + hh) * kRows * kDC + tid;
        r[kReadK * kDC] = rd[tid] * fac[0][tid];
        r[kFk * kDC] = fac[0][tid];
        r[kWriteK * kDC] = wr[tid] * fac[0][tid];
        r[kReadQ * kDC] = a.scale * rd[tid] * fac[1][tid];
        r[kFq * kDC] = a.scale * fac[1][tid];
        r[kBeta * kDC] = bet[tid];
        if constexpr (GRAD) {
            float *e = a.rows2 + (ci * a.h + hh) * kRowsGrad * kDC + tid;
            e[kGhi * kDC] = ghi[tid];
            e[kGlo * kDC] = glo[tid];
            e[kDoc * kDC] = (float)doc[tid];
            e[kRead * kDC] = rd[tid];
            e[kWrite * kDC] = wr[tid];
            e[kRk * kDC] = rn[0][tid];
            e[kRq * kDC] = rn[1][tid];
            e[kStep * kDC] = step;
        }
    }

    // row tile `wave` of K K^T and Q K^T, decayed and masked
    for (int jt = 0; jt <= wave; ++jt) {
        f32x4 kk = zero4(), qk = zero4();
#pragma unroll
        for (int kb = 0; kb < XB; ++kb) {
            const f16x8 kj = img_rows(kq[0], jt * XB + kb, lane);
            const f16x8 ki = img_rows(kq[0], wave * XB + kb, lane);
            const f16x8 qi = img_rows(kq[1], wave * XB + kb, lane);
            kk = mma16(ki, kj, kk);
            qk = mma16(qi, kj, qk);
            if constexpr (F32) {
                const f16x8 lj = img_rows(kq[0] + IMG, jt * XB + kb, lane);
                kk = mma16(ki, lj, kk);
                qk = mma16(qi, lj, qk);
                kk = mma16(img_rows(kq[0] + IMG, wave * XB + kb, lane), kj, kk);
                qk = mma16(img_rows(kq[1] + IMG, wave * XB + kb, lane), kj, qk);
            }
        }
        const int j = 16 * jt + j16;
        const float hj = ghi[j], lj = glo[j], fj = fac[0][j];
        const int dj = doc[j];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * wave + 4 * g + r;
            const bool in = j <= i && doc[i] == dj;
            const float d = in ? exp2f((ghi[i] - hj) + (glo[i] - lj)) : 0.f;
            tri[0][i * kTP + j] = j < i ? kk[r] * d * (fac[0][i] * fj) : 0.f;
            const float p = qk[r] * d;
            const f16 h = (f16)p;
            const int at = tri_piece(wave, jt >> 1) * 512 + (4 * g + r + 16 * (j16 >> 2)) * 8 +
                           4 * (jt & 1) + (j16 & 3);
            pst[0][at] = h;
            if constexpr (PPL == 2) pst[1][at] = (f16)(p - (float)h);
        }
    }
    __syncthreads();

    // the inverses' diagonal blocks: column j16, lane group 0 of T, group 1 of
    // (I + beta kk)^-1
    if (g < NT) {
        float x[16];
        const float *K = tri[0] + 16 * wave * kTP + 16 * wave;
        const float *be = bet + 16 * wave;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < i; ++k) s = fmaf(K[i * kTP + k], g == 0 ? be[k] * x[k] : x[k], s);
            x[i] = (i == j16 ? 1.f : 0.f) - (g == 0 ? s : be[i] * s);
        }
        float *o = (NT == 1 || g == 0 ? tri[1] : tri[NT]) + 16 * wave * kTP + 16 * wave + j16;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i * kTP] = x[i];
    }
    __syncthreads();
    for (int d = 1; d < 4; ++d) {
        for (int task = wave; task < NT * (4 - d); task += 4) {
            const int m = task / (4 - d), j = task % (4 - d), i = j + d;
            float *T = tri[1 + m];
            f32x4 x = zero4();
            for (int k = j; k < i; ++k) {
                const f32x4 ka =
                    *reinterpret_cast<const f32x4 *>(tri[0] + (16 * i + j16) * kTP + 16 * k + 4 * g);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int kr = 16 * k + 4 * g + q;
                    const float t = T[kr * kTP + 16 * j + j16];
                    x = Mfma<float>::mma(ka[q], m == 0 ? bet[kr] * t : t, x);
                }
            }
            if (m == 1)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] *= bet[16 * i + 4 * g + r];
            const f32x4 ti =
                *reinterpret_cast<const f32x4 *>(T + (16 * i + j16) * kTP + 16 * i + 4 * g);
            f32x4 o = zero4();
#pragma unroll
            for (int q = 0; q < 4; ++q) o = Mfma<float>::mma(ti[q], x[q], o);
#pragma unroll
            for (int r = 0; r < 4; ++r) T[(16 * i + 4 * g + r) * kTP + 16 * j + j16] = -o[r];
        }
        __syncthreads();
    }

    // images of the triangles
    f16 *tdst = a.timg + (ci * a.h + hh) * (2 * kPieces * 512);
    f16 *mdst = GRAD ? a.mimg + (ci * a.h + hh) * (2 * kPieces * 512) : nullptr;
    for (int i = tid; i < NT * kPieces * 64; i += 256) {
        const int m = i / (kPieces * 64), piece = (i >> 6) % kPieces, ln = i & 63;
        const int rt = piece < 2 ? piece : 2 + ((piece - 2) >> 1), kb = piece < 2 ? 0 : (piece & 1);
        const float *src = tri[1 + m] + (16 * rt + (ln & 15)) * kTP + 32 * kb + 4 * (ln >> 4);
        const f32x4 u = *reinterpret_cast<const f32x4 *>(src);
        const f32x4 w = 2 * kb + 1 <= rt ? *reinterpret_cast<const f32x4 *>(src + 16) : zero4();
        const Split s = split8(u, w, 1.f);
        f16 *dst = (m ? mdst : tdst) + piece * 512 + ln * 8;
        *reinterpret_cast<f16x8 *>(dst) = s.hi;
        *reinterpret_cast<f16x8 *>(dst + kPieces * 512) = s.lo;
    }
    f16 *pdst = a.pimg + (ci * a.h + hh) * (PPL * kPieces * 512);
    for (int i = tid; i < PPL * kPieces * 64; i += 256)
        reinterpret_cast<u32x4 *>(pdst)[i] = reinterpret_cast<const u32x4 *>(&pst[0][0])[i];
}

// --------------------------------------------------------------- forward ---
// One buffer of LDS: images of k and q, T, tril(Q K^T), the row arrays, then
// the 64 rows of v (and of dy) of the workgroup's columns.
template <typename IO, int N, bool GRAD> struct FwdBuf {
    static constexpr int PL = sizeof(IO) == 4 ? 2 : 1;
    static constexpr int PPL = sizeof(IO) == 4 || GRAD ? 2 : 1;
    static constexpr int K = 0, Q = PL * kDC * N * 2, T = 2 * Q, P = T + 2 * kPieces * 1024;
    static constexpr int R = P + PPL * kPieces * 1024, V = R + kRows * kDC * 4;
    static __host__ __device__ int bytes(int cols) {
        return V + (GRAD ? 2 : 1) * kDC * cols * (int)sizeof(IO);
    }
};

template <typename IO, int N, bool GRAD>
__device__ __forceinline__ void fwd_copy(const DeltaArgs &a, uint32_t buf, int64_t bb, int64_t c,
                                         int64_t hh, int col0, int cols, int wave, int nw, int lane) {
    typedef FwdBuf<IO, N, GRAD> B;
    const int64_t ci = bb * a.nc + c, gi = ci * a.g + hh / (a.h / a.g), hi = ci * a.h + hh;
    const int64_t t0 = c * kDC;
    const int len = (int)(a.l - t0 < kDC ? a.l - t0 : kDC);
    copy_lds(a.kimg + gi * (B::PL * kDC * N), B::Q, B::Q, buf + B::K, wave, nw, lane);
    copy_lds(a.qimg + gi * (B::PL * kDC * N), B::Q, B::Q, buf + B::Q, wave, nw, lane);
    copy_lds(a.timg + hi * (2 * kPieces * 512), 2 * kPieces * 1024, 2 * kPieces * 1024, buf + B::T, wave, nw, lane);
    copy_lds(a.pimg + hi * (B::PPL * kPieces * 512), B::PPL * kPieces * 1024, B::PPL * kPieces * 1024, buf + B::P, wave, nw, lane);
    copy_lds(a.rows + hi * (kRows * kDC), kRows * kDC * 4, kRows * kDC * 4, buf + B::R, wave, nw, lane);
    const int64_t at = ((bb * a.l + t0) * a.h + hh) * a.p + col0;
    const int64_t pitch = a.h * a.p * (int64_t)sizeof(IO);
    copy_rows(static_cast<const IO *>(a.v) + at, pitch, cols * (int)sizeof(IO), len, buf + B::V, wave,
              nw, lane);
    if constexpr (GRAD)
        copy_rows(static_cast<const IO *>(a.dy) + at, pitch, cols * (int)sizeof(IO), len,
                  buf + B::V + kDC * cols * (int)sizeof(IO), wave, nw, lane);
}

// SERIAL: a workgroup walks all chunks of a head's columns; otherwise each
// chunk has a workgroup of its own, started from the kept states (gradient).
template <typename IO, int N, bool GRAD, bool SERIAL, int NB>
__global__ __launch_bounds__(512) void k_delta_fwd(DeltaArgs a) {
    typedef FwdBuf<IO, N, GRAD> B;
    constexpr bool F32 = sizeof(IO) == 4, FULL = F32 || GRAD;
    constexpr int XB = N / 32, NT = N / 16, IMG = kDC * N;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int g = lane >> 4, j16 = lane & 15;
    const int cols = 16 * nw, slices = a.p / cols;
    int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int col0 = (int)(item % slices) * cols;
    item /= slices;
    const int64_t hh = item % a.h;
    item /= a.h;
    const int64_t c0 = SERIAL ? 0 : item % a.nc, bb = SERIAL ? item : item / a.nc;
    const int64_t c1 = SERIAL ? a.nc : c0 + 1;
    const int col = col0 + 16 * wave, ct = col >> 4;
    const int bufbytes = B::bytes(cols);
    const uint32_t base = lds_address(lds);

    fwd_copy<IO, N, GRAD>(a, base, bb, c0, hh, col0, cols, wave, nw, lane);
    f32x4 S[NT];
    {
        const float *src = nullptr;
        if (SERIAL || c0 == 0) {
            if (a.init) src = a.init + (bb * a.h + hh) * N * a.p;
        } else {
            src = a.kept + ((bb * a.nc + c0 - 1) * a.h + hh) * N * a.p;
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            S[x] = zero4();
            if (src)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[x][r] = src[(16 * x + 4 * g + r) * a.p + col + j16];
        }
    }
    for (int64_t c = c0; c < c1; ++c) {
        const char *buf = lds + (NB == 2 ? (c & 1) * bufbytes : 0);
        // the copies of this chunk are older than the last chunk's stores
        if (c == c0)
            vm_wait<0>();
        else if (NB == 1)
            vm_wait<0>();
        else if (!GRAD)
            a.states ? vm_wait<16 + 4 * NT>() : vm_wait<16>();
        else
            vm_wait<(F32 ? 2 * XB : XB) + 4 + 4 + 4 * NT>();
        lds_barrier();
        if (NB == 2 && c + 1 < c1)
            fwd_copy<IO, N, GRAD>(a, base + ((c + 1) & 1) * bufbytes, bb, c + 1, hh, col0, cols, wave,
                                  nw, lane);
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
            if constexpr (GRAD) {  // the state in front, as the gradient's operand
                typedef typename Frag8<IO>::type F;
                F f;
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = (IO)S[2 * kb + (e >> 2)][e & 3];
                reinterpret_cast<F *>(static_cast<IO *>(a.simg) +
                                      (hi * (a.p >> 4) + ct) * (XB * 512))[64 * kb + lane] = f;
            }
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
        f32x4 U[4], W[4];
        mx = 0.f;
        f32x4 Nv[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            f32x4 t = zero4();
#pragma unroll
            for (int tb = 0; tb <= rt / 2; ++tb) {
                const f16x8 th = img_rows(T, tri_piece(rt, tb), lane);
                t = mma16(th, rf[tb].hi, t);
                t = mma16(th, rf[tb].lo, t);
                t = mma16(img_rows(T + kPieces * 512, tri_piece(rt, tb), lane), rf[tb].hi, t);
            }
            const f32x4 be = row4(rows, kBeta, rt, lane), fk = row4(rows, kFk, rt, lane),
                        wk = row4(rows, kWriteK, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = t[r] * pr.inv;
                Nv[rt][r] = v;
                U[rt][r] = v * be[r] * fk[r];
                W[rt][r] = v * be[r] * wk[r];
            }
            mx = abs_max(mx, U[rt]);
        }
        // e^{G_C - G} <= 1, so one power of two serves both
        const Pow2 pu(col_max(mx));
        const float carry = rows[kCarry * kDC];
        if (SERIAL) {
            Split wf[2];
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) wf[tb] = split8(W[2 * tb], W[2 * tb + 1], pu.sc);
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
                for (int r = 0; r < 4; ++r) S[x][r] = fmaf(t[r], pu.inv, carry * S[x][r]);
            }
        }
        // Y = scale (e^G Q S + tril(Q K^T) U)
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
                if constexpr (FULL) t = mma16(q, sf[kb].lo, t);
                if constexpr (F32) t = mma16(img_rows(Q + IMG, rt * XB + kb, lane), sf[kb].hi, t);
            }
#pragma unroll
            for (int tb = 0; tb <= rt / 2; ++tb) {
                const f16x8 p = img_rows(P, tri_piece(rt, tb), lane);
                u = mma16(p, uf[tb].hi, u);
                if constexpr (FULL) {
                    u = mma16(p, uf[tb].lo, u);
                    u = mma16(img_rows(P + kPieces * 512, tri_piece(rt, tb), lane), uf[tb].hi, u);
                }
            }
            const f32x4 fr = row4(rows, kReadQ, rt, lane), fp = row4(rows, kFq, rt, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                Y[rt][r] = fmaf(fr[r] * ps.inv, t[r], fp[r] * pu.inv * u[r]);
        }
        if constexpr (!GRAD) {
            const uint32_t pitch = (uint32_t)(a.h * a.p * sizeof(IO));
            const Rsrc ry = make_rsrc(static_cast<IO *>(a.y) +
                                          ((bb * a.l + t0) * a.h + hh) * a.p + col,
                                      (int64_t)(len - 1) * pitch + 16 * sizeof(IO));
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    buf_put(ry, (16 * rt + 4 * g + r) * pitch + j16 * sizeof(IO), Y[rt][r], IO{});
        } else {
            // N, as the gradient's operand type, in fragment order; with bf16 the
            // remainder too, for dbeta
            typedef typename Frag8<IO>::type F;
            const int64_t at = (hi * (a.p >> 4) + ct) * (2 * 512) + 8 * lane;
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                F f, low;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = Nv[2 * tb + (e >> 2)][e & 3];
                    f[e] = (IO)v;
                    if constexpr (!F32) low[e] = (IO)(v - (float)f[e]);
                }
                *reinterpret_cast<F *>(static_cast<IO *>(a.nimg) + at + 512 * tb) = f;
                if constexpr (!F32) *reinterpret_cast<F *>(static_cast<IO *>(a.nlow) + at + 512 * tb) = low;
            }
            const IO *dY = V + kDC * cols;
            float *o = a.doo + (hi * (a.p >> 4) + ct) * kDC;
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                f32x4 d = lds_tile(dY, cols, rt, 16 * wave, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) d[r] = sum16(d[r] * Y[rt][r]);
                if (j16 == 0) *reinterpret_cast<f32x4 *>(o + 16 * rt + 4 * g) = d;
            }
        }
        if (SERIAL && a.states) {
            float *st = a.states + hi * N * a.p + col;
            const Rsrc rs = make_rsrc(st, ((int64_t)(N - 1) * a.p + 16) * 4);
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    buf_put(rs, (uint32_t)(((16 * x + 4 * g + r) * a.p + j16) * 4), S[x][r], 0.f);
        }
        if (NB == 1 && c + 1 < c1) {
            lds_barrier();  // everyone is done with the buffer
            fwd_copy<IO, N, GRAD>(a, base, bb, c + 1, hh, col0, cols, wave, nw, lane);
        }
    }
    if (SERIAL && a.fin) {
        float *dst = a.fin + (bb * a.h + hh) * N * a.p + col + j16;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(16 * x + 4 * g + r) * a.p] = S[x][r];
    }
}

constexpr int kLdsMost = 160 * 1024;

template <typename IO, int N, bool GRAD, bool SERIAL>
hipError_t run_fwd(const DeltaArgs &a, hipStream_t s) {
    typedef FwdBuf<IO, N, GRAD> B;
    // columns of a workgroup: all of a head's where that still gives every
    // compute unit a workgroup (its images are then copied once), else 64
    int nw = a.p / 16;
    if (nw > 4 && a.b * a.h * (SERIAL ? 1 : a.nc) < device_cus()) nw = 4;
    if (!SERIAL && nw > 4) nw = 4;
    const int one = B::bytes(16 * nw);
    const int64_t items = a.b * a.h * (a.p / (16 * nw)) * (SERIAL ? 1 : a.nc);
    const dim3 grid((unsigned)items), block(64 * nw);
    if (SERIAL && 2 * one <= kLdsMost) {
        auto *k = &k_delta_fwd<IO, N, GRAD, SERIAL, 2>;
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLdsMost);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k, grid, block, 2 * one, s, a);
    } else {
        auto *k = &k_delta_fwd<IO, N, GRAD, SERIAL, 1>;
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLdsMost);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k, grid, block, one, s, a);
    }
    return hipGetLastError();
}

template <typename IO, int N> hipError_t prep_n(const DeltaArgs &a, bool grad, hipStream_t s) {
    const dim3 grid((unsigned)(a.b * a.nc * a.h)), block(256);
    if (grad)
        hipLaunchKernelGGL((k_delta_prep<IO, N, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_delta_prep<IO, N, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <typename IO, int N> hipError_t fwd_n(const DeltaArgs &a, bool grad, hipStream_t s) {
    if (!grad) return run_fwd<IO, N, false, true>(a, s);
    return a.kept ? run_fwd<IO, N, true, false>(a, s) : run_fwd<IO, N, true, true>(a, s);
}

}  // namespace

hipError_t delta_prep(const DeltaArgs &a, int io, int n, bool grad, hipStream_t s) {
    if (io == SSD_BF16)
        return n == 32 ? prep_n<bf16, 32>(a, grad, s)
                       : n == 64 ? prep_n<bf16, 64>(a, grad, s) : prep_n<bf16, 128>(a, grad, s);
    return n == 32 ? prep_n<float, 32>(a, grad, s)
                   : n == 64 ? prep_n<float, 64>(a, grad, s) : prep_n<float, 128>(a, grad, s);
}

hipError_t delta_forward(const DeltaArgs &a, int io, int n, bool grad, hipStream_t s) {
    if (io == SSD_BF16)
        return n == 32 ? fwd_n<bf16, 32>(a, grad, s)
                       : n == 64 ? fwd_n<bf16, 64>(a, grad, s) : fwd_n<bf16, 128>(a, grad, s);
    return n == 32 ? fwd_n<float, 32>(a, grad, s)
                   : n == 64 ? fwd_n<float, 64>(a, grad, s) : fwd_n<float, 128>(a, grad, s);
}

}  // namespace ssd
