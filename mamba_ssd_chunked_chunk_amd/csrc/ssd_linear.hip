// The products around the mixer: out = act(x W^T + bias) + residual, and its
// gradient dx = e W, dW = e^T x, dbias = sum e with e = dy act'(pre).
//
// Every product is D[m][n] = sum_k A(m, k) B(n, k) on the matrix cores with
// fp32 accumulation.  An operand is stored with its contraction index
// contiguous (rows [m][k], read from LDS 16 bytes a lane) or outermost
// ([k][m], read from LDS through the transposing loads); the forward product
// has both operands the first way, dx has W the second way, dW both.
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "../../include/ssd.h"
#include "ssd_copies.hpp"
#include "ssd_device.hpp"

namespace ssd {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
// Whether p is aligned as rows of `width` elements are among themselves: to the
// largest power of two up to 16 that divides a row's bytes.
bool row_al(const void *p, int64_t width, int64_t es) {
    const int64_t low = (width * es) & -(width * es);
    return al(p, low < 16 ? low : 16);
}

// ---------------------------------------------------------- activations ----
// The normal distribution's Phi(v) = (1 + erf(v / sqrt 2)) / 2 for GELU, with the
// exponential e = e^{-v^2/2} that its density shares:  Phi(-z) = e R(t), t =
// 1 / (1 + z / 4), where R is the polynomial of degree 7 without constant term of
// least largest |e dR|: with these coefficients as fp32 holds them 1.7e-8, against
// 6e-8 for one rounding of Phi, and in relation to Phi(-z) 1.7e-6 up to z = 3,
// 1.2e-5 up to 8 and 3e-5 up to 14.  With the library's erf the gradient's
// preparation was bound by vector issue (93% busy; 67 against 56 us, traced).
__device__ __forceinline__ float normal_cdf(float v, float &e) {
    const float z = fabsf(v), t = __builtin_amdgcn_rcpf(fmaf(0.25f, z, 1.f));
    float r = fmaf(t, -0.09097318566f, 0.3389475501f);
    r = fmaf(t, r, -0.2624053838f);
    r = fmaf(t, r, 0.2770758760f);
    r = fmaf(t, r, 0.02676932733f);
    r = fmaf(t, r, 0.1117260341f);
    r = fmaf(t, r, 0.09885979029f);
    e = exp2_fast(-0.5f * kLog2e * v * v);
    const float q = e * (r * t);
    return v < 0.f ? q : 1.f - q;
}

__device__ __forceinline__ float act_f(float v, int act) {
    float e;
    if (act == SSD_ACT_SILU) return v * __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
    if (act == SSD_ACT_GELU) return v * normal_cdf(v, e);
    if (act == SSD_ACT_SIGMOID) return __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
    return v;
}
__device__ __forceinline__ float act_grad(float v, int act) {
    if (act == SSD_ACT_GELU) {
        float e;
        const float p = normal_cdf(v, e);
        return fmaf(0.3989422804014327f * v, e, p);
    }
    const float s = __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
    if (act == SSD_ACT_SILU) return s * (1.f + v * (1.f - s));
    if (act == SSD_ACT_SIGMOID) return s * (1.f - s);
    return 1.f;
}

// -------------------------------------------------------------- operands ----
// One 16-byte piece per lane is 8 bf16 or 4 fp32 of the contraction: one
// 16x16x32 product, or four 16x16x4 products whose step s takes element s of
// every lane's piece (both operands alike, so the sum is whole).
template <typename IO> struct Mma;
template <> struct Mma<bf16> {
    static __device__ __forceinline__ f32x4 go(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <> struct Mma<float> {
    static __device__ __forceinline__ f32x4 go(u32x4 a, u32x4 b, f32x4 c) {
        const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s], y[s], c, 0, 0, 0);
        return c;
    }
};

// What becomes of a product's elements.
struct Epi {
    void *out;           // [m][n]
    const float *bias;   // [n] or NULL
    const void *res;     // [m][n] or NULL
    void *pre;           // [m][n] or NULL
    int act;
};

struct GemmArgs {
    const void *A, *B;
    int64_t lda, ldb;    // elements per stored row
    int64_t m, n, k;
    int64_t tm, tn;      // tiles
    int64_t split, kper; // contraction parts, elements per part (a multiple of the step)
    float *parts;        // [split][m][n] where split > 1
    Epi ep;
};

// Four consecutive elements as fp32, and back, at any element alignment (rows
// of odd widths; the memory takes vector accesses there too).
__device__ __forceinline__ f32x4 ldu4(const float *p) {
    f32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ f32x4 ldu4(const bf16 *p) {
    bf16x4 v;
    __builtin_memcpy(&v, p, 8);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ void stu4(float *p, f32x4 v) { __builtin_memcpy(p, &v, 16); }
__device__ __forceinline__ void stu4(bf16 *p, f32x4 v) {
    bf16x4 o;
    o[0] = (bf16)v[0]; o[1] = (bf16)v[1]; o[2] = (bf16)v[2]; o[3] = (bf16)v[3];
    __builtin_memcpy(p, &o, 8);
}

template <typename IO> struct Four { typedef f32x4 type; };
template <> struct Four<bf16> { typedef bf16x4 type; };

// Four consecutive n of one row m.
template <typename IO>
__device__ __forceinline__ void finish4(const Epi &ep, int64_t m, int64_t n, int64_t N, f32x4 v) {
    const int64_t at = m * N + n;
    if (n + 4 <= N) {
        if (ep.bias) v += ldu4(ep.bias + n);
        if (ep.pre) stu4(static_cast<IO *>(ep.pre) + at, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_f(v[i], ep.act);
        if (ep.res) v += ldu4(static_cast<const IO *>(ep.res) + at);
        stu4(static_cast<IO *>(ep.out) + at, v);
        return;
    }
    for (int i = 0; n + i < N; ++i) {
        float x = i == 0 ? v[0] : i == 1 ? v[1] : v[2];
        if (ep.bias) x += ep.bias[n + i];
        if (ep.pre) static_cast<IO *>(ep.pre)[at + i] = (IO)x;
        x = act_f(x, ep.act);
        if (ep.res) x += to_f32(static_cast<const IO *>(ep.res)[at + i]);
        static_cast<IO *>(ep.out)[at + i] = (IO)x;
    }
}

// ------------------------------------------------------------ LDS tiles ----
template <typename IO, bool TR, int BM> using OpTile = TileGeometry<(int)sizeof(IO), TR, BM>;

// A wave's share of an operand's copies into LDS, a step of the contraction at
// a time: byte offsets from the step's first element, the same in every step,
// and the resource that the step reads through, moved on by one scalar
// addition.
template <typename IO, bool TR, int BM, int NT> struct Copies {
    typedef OpTile<IO, TR, BM> T;
    static constexpr int N = T::BYTES / 16 / NT;
    static_assert(T::BYTES % (16 * NT) == 0, "every wave copies as much");
    const CopySteps<(int)sizeof(IO), TR, BM> plan;
    uint32_t off[N];
    const char *base;
    __device__ __forceinline__ Copies(const void *src, int64_t ld, int64_t m0, int64_t mEnd,
                                      int64_t k0, int64_t kEnd, int steps)
        : plan(ld, m0, mEnd, k0, kEnd, steps), base(static_cast<const char *>(src) + plan.first) {
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = T::offset(i * NT + (int)threadIdx.x, ld);
    }
    __device__ __forceinline__ void next(char *lds, bool final) {
        const RsrcW r = make_rsrc_w(base, final ? plan.last : plan.bytes);
        char *dst = lds + wave_id() * 1024;
        if (!TR && final && plan.tail < T::BK) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                lds_dma16(r, (lds_void *)(dst + i * NT * 16),
                          plan.masked(i * NT + (int)threadIdx.x) ? 0xffffff00u : off[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) lds_dma16(r, (lds_void *)(dst + i * NT * 16), off[i]);
        }
        base += plan.stride;
    }
};

// The 16-byte operand piece of lane l: tile row m = r0 + (l & 15), contraction
// chunk 4 j + (l >> 4) of the step.
template <typename IO, bool TR, int BM>
__device__ __forceinline__ u32x4 piece(const char *lds, int r0, int j, int lane) {
    typedef OpTile<IO, TR, BM> T;
    const int c = lane & 15, q = 4 * j + (lane >> 4);
    if constexpr (!TR) {
        const int row = r0 + c;
        return *reinterpret_cast<const u32x4 *>(lds + (row * T::CH + (q ^ T::f(row))) * 16);
    } else if constexpr (sizeof(IO) == 2) {
        const int ka = q * 8 + (c >> 2), col = r0 + 4 * (c & 3);
        auto at = [&](int k) {
            return lds + (k * T::CH + ((col >> 3) ^ T::f(k))) * 16 + (col & 7) * 2;
        };
        const f16x4 a = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)at(ka)));
        const f16x4 b = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4 *)at(ka + 4)));
        return __builtin_bit_cast(u32x4, f16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    } else {
        const int col = r0 + c;
        u32x4 v;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = q * 4 + s;
            v[s] = *reinterpret_cast<const uint32_t *>(
                lds + (k * T::CH + ((col >> 2) ^ T::f(k))) * 16 + (col & 3) * 4);
        }
        return v;
    }
}

constexpr uint32_t kBand = 8;

// One workgroup: a BM x BN tile of D over one contraction part, WM x WN waves,
// two steps of both operands in LDS, copied there without registers.
//
// A step waits for its own copies and for everyone, starts the next step's
// copies and multiplies.  What hides its waits is the other workgroup of the
// compute unit, not a deeper pipeline: at 16384 x 5120 -> 2560 (bf16) a
// 256 x 256 tile (one workgroup a unit, 8 waves) took 470 us, 256 x 320 440,
// 128 x 128 422 with 4 waves and 398 with 8, and 128 x 192 with 8 waves, whose
// two workgroups fill the 160 KB of LDS, 376 (as first measured, side by side;
// as it stands 385, 1117 TFLOP/s, and 397 to 426 with the residual, by the box).
// Three or four steps in flight changed nothing, nor did reading operand pieces
// ahead.  L2 gives 17 TB/s (a 128-byte request each 2 clocks and channel), 1320
// TFLOP/s for this tile's 77 operations a byte: that and the last, partly filled
// round are what it is bound by.
template <typename IO, bool TA, bool TB, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void gemm_tile(const GemmArgs &g, uint32_t item, char *lds) {
    constexpr int NT = WM * WN * 64;
    typedef OpTile<IO, TA, BM> OA;
    typedef OpTile<IO, TB, BN> OB;
    constexpr int BK = OA::BK, SIZE = OA::BYTES + OB::BYTES;
    constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    const int lane = threadIdx.x & 63, wv = wave_id();
    const uint32_t tn = (uint32_t)g.tn, all = (uint32_t)g.tm * tn;
    const uint32_t part = item / all, tile = item % all;
    // tiles in bands of kBand tile rows, down the rows first: the tiles that run
    // at one time on an XCD (consecutive items) share rows of both operands
    const uint32_t band = tile / (kBand * tn), in = tile % (kBand * tn);
    const uint32_t left = (uint32_t)g.tm - band * kBand, rows = left < kBand ? left : kBand;
    const int64_t m0 = (int64_t)(band * kBand + in % rows) * BM, n0 = (int64_t)(in / rows) * BN;
    const int64_t k0 = part * g.kper, kEnd = k0 + g.kper < g.k ? k0 + g.kper : g.k;
    const int wm = wv / WN * (BM / WM), wn = wv % WN * (BN / WN);
    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = zero4();
    const int steps = (int)((kEnd - k0 + BK - 1) / BK);
    Copies<IO, TA, BM, NT> ca(g.A, g.lda, m0, g.m, k0, kEnd, steps);
    Copies<IO, TB, BN, NT> cb(g.B, g.ldb, n0, g.n, k0, kEnd, steps);
    auto copy = [&](int slot, bool final) {
        ca.next(lds + slot * SIZE, final);
        cb.next(lds + slot * SIZE + OA::BYTES, final);
    };
    // One step from the LDS slot it was copied to, while the next is copied to
    // the other one: this step's copies have landed, and everyone has read the
    // step before.
    auto step = [&](int k, auto s) {
        constexpr int slot = decltype(s)::value;
        vm_wait<0>();
        lds_barrier();
        if (k + 1 < steps) copy(1 - slot, k + 2 == steps);
        const char *a = lds + slot * SIZE, *b = a + OA::BYTES;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            u32x4 pa[MI], pb[NI];
#pragma unroll
            for (int i = 0; i < MI; ++i) pa[i] = piece<IO, TA, BM>(a, wm + 16 * i, j, lane);
#pragma unroll
            for (int i = 0; i < NI; ++i) pb[i] = piece<IO, TB, BN>(b, wn + 16 * i, j, lane);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int n = 0; n < NI; ++n) acc[i][n] = Mma<IO>::go(pb[n], pa[i], acc[i][n]);
        }
    };
    copy(0, steps == 1);
    for (int k = 0; k < steps; k += 2) {
        step(k, std::integral_constant<int, 0>{});
        if (k + 1 < steps) step(k + 1, std::integral_constant<int, 1>{});
    }
    // element r of a lane: row m of lane & 15, column 4 (lane >> 4) + r
    const int64_t mw = m0 + wm + (lane & 15), nw = n0 + wn + 4 * (lane >> 4);
    if (g.split > 1) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int64_t m = mw + 16 * i, n = nw + 16 * j;
                if (m >= g.m || n >= g.n) continue;
                float *p = g.parts + (part * g.m + m) * g.n + n;
                if (n + 4 <= g.n)
                    stu4(p, acc[i][j]);
                else
                    for (int r = 0; n + r < g.n; ++r) p[r] = acc[i][j][r];
            }
    } else if (m0 + wm + BM / WM <= g.m && n0 + wn + BN / WN <= g.n) {
        // the wave's part is whole: every residual and bias is requested before
        // any is used (one after the other, each element waited for its own)
        const int64_t at = mw * g.n + nw;
        typedef typename Four<IO>::type R;
        R res[MI][NI];
        f32x4 bias[NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) bias[j] = g.ep.bias ? ldu4(g.ep.bias + nw + 16 * j) : zero4();
        if (g.ep.res) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    __builtin_memcpy(&res[i][j],
                                     static_cast<const IO *>(g.ep.res) + at + 16 * i * g.n + 16 * j,
                                     sizeof(R));
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int64_t to = at + 16 * i * g.n + 16 * j;
                f32x4 v = acc[i][j] + bias[j];
                if (g.ep.pre) stu4(static_cast<IO *>(g.ep.pre) + to, v);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = act_f(v[r], g.ep.act);
                if (g.ep.res) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] += (float)res[i][j][r];
                }
                stu4(static_cast<IO *>(g.ep.out) + to, v);
            }
    } else {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int64_t m = mw + 16 * i, n = nw + 16 * j;
                if (m < g.m && n < g.n) finish4<IO>(g.ep, m, n, g.n, acc[i][j]);
            }
    }
}

template <typename IO, bool TA, bool TB, int BM, int BN> constexpr int lds_bytes() {
    return 2 * (OpTile<IO, TA, BM>::BYTES + OpTile<IO, TB, BN>::BYTES);
}

// The forward product.
template <typename IO, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void k_gemm(GemmArgs g) {
    __shared__ __align__(16) char lds[lds_bytes<IO, false, false, BM, BN>()];
    gemm_tile<IO, false, false, BM, BN, WM, WN>(
        g, (uint32_t)xcd_item(blockIdx.x, gridDim.x), lds);
}

// The gradient's two products in one launch: dx = e W and dW = e^T x, the one
// with the longer contraction first so that the other fills the last round.
// Each is dealt over all XCDs by itself: one run of items over both would give
// some XCDs only long ones (477 against 385 us for 8192 x 2560 -> 5120).
template <typename IO, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void k_gemm_bwd(GemmArgs gx, GemmArgs gw, int wfirst) {
    __shared__ __align__(16) char lds[lds_bytes<IO, true, true, BM, BN>()];
    const uint32_t nx = (uint32_t)(gx.tm * gx.tn * gx.split), nw = (uint32_t)(gw.tm * gw.tn * gw.split);
    const uint32_t lead = wfirst ? nw : nx, b = blockIdx.x;
    const bool w = (b < lead) == (wfirst != 0);
    const uint32_t item = (uint32_t)xcd_item(b < lead ? b : b - lead, w ? nw : nx);
    if (w)
        gemm_tile<IO, true, true, BM, BN, WM, WN>(gw, item, lds);
    else
        gemm_tile<IO, false, true, BM, BN, WM, WN>(gx, item, lds);
}

// Four consecutive elements of a product in parts: their sum in the parts'
// order, and what follows it.
template <typename IO> __device__ __forceinline__ void sum_parts(const GemmArgs &g, uint32_t k) {
    const uint32_t q = (uint32_t)((g.n + 3) / 4);
    const int64_t row = k / q, col = (int64_t)(k % q) * 4;
    f32x4 v = zero4();
    for (int64_t s = 0; s < g.split; ++s) {
        const float *p = g.parts + (s * g.m + row) * g.n + col;
        if (col + 4 <= g.n)
            v += ldu4(p);
        else
            for (int r = 0; r < 4 && col + r < g.n; ++r) v[r] += p[r];
    }
    finish4<IO>(g.ep, row, col, g.n, v);
}
template <typename IO> __global__ __launch_bounds__(256) void k_gemm_sum(GemmArgs g) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k < g.m * ((g.n + 3) / 4)) sum_parts<IO>(g, (uint32_t)k);
}

// ------------------------------------------------------------- few rows ----
// Up to 16 MT rows of x (decoded tokens): bound by the weight's bytes.  A
// workgroup owns 16 weight rows, its waves 128-byte pieces of them in turn,
// loaded from memory straight into operands (at any alignment: rows of odd
// widths are read where they are); the waves' sums meet in LDS and are added
// in order.  One row, 2560 -> 10576 bf16: 11.9 us, 4.5 TB/s of weight (4 waves;
// 8 leave 21 of the 661 workgroups to a second round, 15.0 us, 16 waves 22 us).
// 32 rows of 768 -> 3352: 4.8 us (see few_fwd for what the tiles take).
constexpr int kFewWaves = 4;
constexpr int kFewUnroll = 4;  // weight pieces in flight a wave

// The 16 bytes of a row of `width` elements from element c, zeros past its end.
template <typename IO> __device__ __forceinline__ u32x4 row16(const IO *row, int64_t c, int64_t width) {
    constexpr int N = 16 / (int)sizeof(IO);
    u32x4 v = {0, 0, 0, 0};
    if (c + N <= width) {
        __builtin_memcpy(&v, row + c, 16);
    } else if (c < width) {
        IO e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = c + i < width ? row[c + i] : (IO)0.f;
        __builtin_memcpy(&v, e, 16);
    }
    return v;
}

template <typename IO, int MT>
__global__ __launch_bounds__(kFewWaves * 64) void k_few(GemmArgs g) {
    constexpr int EPC = 16 / (int)sizeof(IO), BK = 8 * EPC;
    __shared__ f32x4 part[kFewWaves][MT][64];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int c = lane & 15, q = lane >> 4;
    const int64_t nr = n0 + c < g.n ? n0 + c : g.n - 1;
    const IO *w = static_cast<const IO *>(g.B) + nr * g.ldb;
    const IO *x[MT];
    bool live[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        live[t] = t * 16 + c < g.m;
        x[t] = static_cast<const IO *>(g.A) + (live[t] ? t * 16 + c : 0) * g.lda;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = zero4();
    const u32x4 none = {0, 0, 0, 0};
    auto steps = [&](int64_t k, auto whole) {
        u32x4 pw[2 * kFewUnroll], px[2 * kFewUnroll][MT];
#pragma unroll
        for (int i = 0; i < 2 * kFewUnroll; ++i) {
            const int64_t at = k + i / 2 * (kFewWaves * BK) + (4 * (i & 1) + q) * EPC;
            constexpr bool W = decltype(whole)::value;
            if (W)
                __builtin_memcpy(&pw[i], w + at, 16);
            else
                pw[i] = row16(w, at, g.k);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (W)
                    __builtin_memcpy(&px[i][t], x[t] + at, 16);
                else
                    px[i][t] = row16(x[t], at, g.k);
                if (!live[t]) px[i][t] = none;
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * kFewUnroll; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[t] = Mma<IO>::go(pw[i], px[i][t], acc[t]);
    };
    constexpr int64_t RUN = (int64_t)kFewUnroll * kFewWaves * BK;
    for (int64_t k = wv * BK; k < g.k; k += RUN) {
        if (k + RUN <= g.k)
            steps(k, std::true_type{});
        else
            steps(k, std::false_type{});
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wv][t][lane] = acc[t];
    __syncthreads();
    if (wv >= MT) return;
    f32x4 v = part[0][wv][lane];
#pragma unroll
    for (int k = 1; k < kFewWaves; ++k) v += part[k][wv][lane];
    const int64_t m = wv * 16 + c, n = n0 + 4 * q;
    if (m < g.m && n < g.n) finish4<IO>(g.ep, m, n, g.n, v);
}

// ------------------------------------------------------------ gradient ----
// Everything before the gradient's products in one launch, in 8-element pieces
// of rows (rows of odd widths start at any element; the memory takes vector
// accesses there too): e = dy act'(pre), with its fp32 column sums over runs
// of `run` rows, and x and W laid out again with padded rows.  Bound by memory:
// 8192 x 5120 bf16 with GELU in 52-56 us, 4.6 TB/s.
//
// With bf16 io e is rounded to bf16, as dy and x are: it is an operand of both
// products, whose other operand is bf16, and the matrix cores take both in one
// type.  In fp32 the two products would run at a ninth of the rate and e would
// be twice the bytes; as a sum of two bf16 values they would be twice the work.  So dx and
// dweight carry two roundings instead of one, independent of each other: against
// fp64 they are off by 0.00235 of their norm (2^-8.7), and by 0.00166 where e is kept
// in fp32.  dbias takes e before the rounding.
struct PrepArgs {
    const void *dy, *pre, *x, *w;
    void *e, *px, *pw;        // NULL: not wanted
    float *part;              // [runs][n] column sums of e, or NULL
    int run;                  // rows of a workgroup: a multiple of 16
    int64_t m, n, k, ln, lk;  // ln, lk: elements per padded row
    int act;
    int64_t eb, xb, wb;       // workgroups of each piece of work
};

template <typename IO> struct alignas(16) Piece { IO v[8]; };

// Elements c .. c + 7 of a row of `width`, zeros past its end.  What lies past
// the row but before `end`, the tensor's end, is read and dropped.
template <typename IO>
__device__ __forceinline__ Piece<IO> row_piece(const IO *row, int64_t c, int64_t width,
                                               const IO *end) {
    Piece<IO> p;
    if (row + c + 8 <= end) {
        __builtin_memcpy(&p, row + c, sizeof(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p.v[i] = c + i < width ? row[c + i] : (IO)0.f;
    }
    if (c + 8 > width) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i >= width) p.v[i] = (IO)0.f;
    }
    return p;
}

// Rows of `cols` elements laid out with `ld` a row (a multiple of 8), zeros
// behind them; workgroup `block` of a grid of them.
template <typename IO>
__device__ __forceinline__ void pad_rows(const void *src, void *dst, int64_t rows, int64_t cols,
                                         int64_t ld, int64_t block) {
    const uint32_t per = (uint32_t)(ld / 8), k = (uint32_t)block * 256 + threadIdx.x;
    if (k >= rows * per) return;
    const int64_t r = k / per, c = (int64_t)(k % per) * 8;
    *reinterpret_cast<Piece<IO> *>(static_cast<IO *>(dst) + r * ld + c) =
        row_piece(static_cast<const IO *>(src) + r * cols, c, cols,
                  static_cast<const IO *>(src) + rows * cols);
}

template <typename IO> __global__ __launch_bounds__(256) void k_pad(PrepArgs g) {
    const int64_t b = blockIdx.x;
    if (b < g.xb)
        pad_rows<IO>(g.x, g.px, g.m, g.k, g.lk, b);
    else
        pad_rows<IO>(g.w, g.pw, g.n, g.k, g.lk, b - g.xb);
}

template <typename IO> __global__ __launch_bounds__(256) void k_bwd_prep(PrepArgs g) {
    __shared__ float sums[4][64 * 8];
    uint32_t b = blockIdx.x;
    if (b >= g.eb) {
        b -= (uint32_t)g.eb;
        if (b < g.xb)
            pad_rows<IO>(g.x, g.px, g.m, g.k, g.lk, b);
        else
            pad_rows<IO>(g.w, g.pw, g.n, g.k, g.lk, b - g.xb);
        return;
    }
    // a wave: 512 columns of a quarter of the run's rows
    const int lane = threadIdx.x & 63, wv = wave_id();
    const uint32_t cols = (uint32_t)((g.ln + 511) / 512);
    const int64_t run = b / cols, c = (int64_t)(b % cols * 64 + lane) * 8;
    constexpr int U = 4;
    const int R = g.run / 4;
    const int64_t r0 = run * g.run + wv * R;
    const IO *dy = static_cast<const IO *>(g.dy), *pre = static_cast<const IO *>(g.pre);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
    if (c < g.ln) {
        for (int64_t r = r0; r < r0 + R && r < g.m; r += U) {
            Piece<IO> d[U], p[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = r + u < g.m ? r + u : g.m - 1;
                d[u] = row_piece(dy + row * g.n, c, g.n, dy + g.m * g.n);
                if (pre) p[u] = row_piece(pre + row * g.n, c, g.n, pre + g.m * g.n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + u >= g.m) break;
                Piece<IO> o;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v = to_f32(d[u].v[i]);
                    if (pre) v *= act_grad(to_f32(p[u].v[i]), g.act);
                    s[i] += v;
                    o.v[i] = (IO)v;
                }
                if (g.e)
                    *reinterpret_cast<Piece<IO> *>(static_cast<IO *>(g.e) + (r + u) * g.ln + c) = o;
            }
        }
    }
    if (!g.part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[wv][i * 64 + lane] = s[i];
    __syncthreads();
    for (int k = threadIdx.x; k < 512; k += 256) {
        const int64_t col = (int64_t)(b % cols) * 512 + (k & 63) * 8 + (k >> 6);
        if (col < g.n)
            g.part[run * g.n + col] = (sums[0][k] + sums[1][k]) + (sums[2][k] + sums[3][k]);
    }
}

// The whole gradient of up to 8 rows in one pass over the weight: bound by its
// bytes, read for dx and written for dW.  A workgroup owns 16 bytes a lane of
// `run` weight rows; its waves take rows in turn.  e is worked out in LDS in
// fp32 (and stays fp32); dx goes out in one part per run, in fp32.  1 row,
// 2560 -> 10576 bf16: 29 us with the sum of the parts (108 MB of weight and
// gradient, 3.7 TB/s), 38 by the tiles.
constexpr int kFewBwdRows = 8, kFewRun = 128;  // rows of x; weight rows of a workgroup at most

template <typename IO, int M>
__global__ __launch_bounds__(256) void k_few_bwd(PrepArgs g, GemmArgs gx, IO *dw, float *db) {
    constexpr int V = 16 / (int)sizeof(IO);
    __shared__ float es[kFewRun][M];
    __shared__ float red[4][64 * V];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const uint32_t cols = (uint32_t)((g.k + 64 * V - 1) / (64 * V));
    const int64_t run = blockIdx.x / cols, c = (int64_t)(blockIdx.x % cols * 64 + lane) * V;
    const int64_t n0 = run * g.run, n1 = n0 + g.run < g.n ? n0 + g.run : g.n;
    const int rows = (int)(n1 - n0);
    const IO *dy = static_cast<const IO *>(g.dy), *pre = static_cast<const IO *>(g.pre);
    for (int i = threadIdx.x; i < rows * M; i += 256) {
        const int m = i / rows, r = i % rows;
        float e = 0.f;
        if (m < g.m) {
            e = to_f32(dy[m * g.n + n0 + r]);
            if (pre) e *= act_grad(to_f32(pre[m * g.n + n0 + r]), g.act);
        }
        es[r][m] = e;
    }
    float x[M][V], dx[M][V];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        u32x4 v = {0, 0, 0, 0};
        if (dw && m < g.m) v = row16(static_cast<const IO *>(g.x) + m * g.k, c, g.k);
        IO e[V];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < V; ++i) x[m][i] = to_f32(e[i]), dx[m][i] = 0.f;
    }
    __syncthreads();
    if (db && blockIdx.x % cols == 0)
        for (int r = threadIdx.x; r < rows; r += 256) {
            float t = 0.f;
#pragma unroll
            for (int m = 0; m < M; ++m) t += es[r][m];
            db[n0 + r] = t;
        }
    constexpr int U = 4;  // weight rows in flight a wave
    for (int r = wv; r < rows; r += 4 * U) {
        u32x4 pw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = r + 4 * u < rows ? r + 4 * u : r;
            pw[u] = u32x4{0, 0, 0, 0};
            if (gx.tm) pw[u] = row16(static_cast<const IO *>(g.w) + (n0 + q) * g.k, c, g.k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = r + 4 * u;
            if (q >= rows) break;
            IO we[V], o[V];
            __builtin_memcpy(we, &pw[u], 16);
            float s[V];
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = 0.f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float e = es[q][m];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] = fmaf(e, x[m][i], s[i]);
                    dx[m][i] = fmaf(e, to_f32(we[i]), dx[m][i]);
                }
            }
            if (!dw || c >= g.k) continue;
            IO *to = dw + (n0 + q) * g.k + c;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = (IO)s[i];
            if (c + V <= g.k)
                __builtin_memcpy(to, o, 16);
            else
                for (int i = 0; i < V; ++i)
                    if (c + i < g.k) to[i] = o[i];
        }
    }
    if (!gx.tm) return;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if (m >= g.m) break;
#pragma unroll
        for (int i = 0; i < V; ++i) red[wv][i * 64 + lane] = dx[m][i];
        __syncthreads();
        for (int k = threadIdx.x; k < 64 * V; k += 256) {
            const int64_t col = (int64_t)(blockIdx.x % cols) * 64 * V + (k & 63) * V + (k >> 6);
            if (col < g.k)
                gx.parts[(run * g.m + m) * g.k + col] =
                    (red[0][k] + red[1][k]) + (red[2][k] + red[3][k]);
        }
        __syncthreads();
    }
}

// dx of few rows from its runs' parts: a workgroup takes 128 columns of a row,
// 8 runs at a time with four loads in flight, added in a fixed order.
template <typename IO> __global__ __launch_bounds__(256) void k_few_sum(GemmArgs g) {
    __shared__ f32x4 s[8][32];
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t row = blockIdx.y, col = ((int64_t)blockIdx.x * 32 + c) * 4;
    auto part = [&](int64_t r) {
        const float *p = g.parts + (r * g.m + row) * g.n + col;
        f32x4 v = zero4();
        if (col + 4 <= g.n)
            v = ldu4(p);
        else
            for (int i = 0; col + i < g.n; ++i) v[i] = p[i];
        return v;
    };
    f32x4 t = zero4();
    int64_t r = q;
    for (; r + 24 < g.split; r += 32) {
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = part(r + 8 * i);
        t += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; r < g.split; r += 8) t += part(r);
    s[q][c] = t;
    __syncthreads();
    if (q != 0 || col >= g.n) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) t += s[k][c];
    finish4<IO>(g.ep, row, col, g.n, t);
}

// Everything after them in one launch: the sums of products in parts, and the
// bias gradient from its runs' sums (a workgroup: 32 columns by 8 runs at a
// time, four loads in flight, added in a fixed order).
template <typename IO>
__global__ __launch_bounds__(256) void k_bwd_finish(GemmArgs gx, GemmArgs gw, int64_t xb, int64_t wb,
                                                    const float *part, int64_t runs, float *db) {
    __shared__ float s[8][32];
    int64_t b = blockIdx.x;
    if (b < xb) {
        const int64_t k = b * 256 + threadIdx.x;
        if (k < gx.m * ((gx.n + 3) / 4)) sum_parts<IO>(gx, (uint32_t)k);
        return;
    }
    b -= xb;
    if (b < wb) {
        const int64_t k = b * 256 + threadIdx.x;
        if (k < gw.m * ((gw.n + 3) / 4)) sum_parts<IO>(gw, (uint32_t)k);
        return;
    }
    b -= wb;
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t col = b * 32 + c, n = gw.m;
    float t = 0.f;
    if (col < n) {
        int64_t r = q;
        for (; r + 24 < runs; r += 32) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = part[(r + 8 * i) * n + col];
            t += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < runs; r += 8) t += part[r * n + col];
    }
    s[q][c] = t;
    __syncthreads();
    if (q != 0 || col >= n) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) t += s[k][c];
    db[col] = t;
}

template <typename IO>
__global__ __launch_bounds__(256) void k_zero(IO *p, int64_t n) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
        p[k] = (IO)0.f;
}

// --------------------------------------------------------------- the plan ----
size_t up(size_t v) { return (v + 255) & ~(size_t)255; }
// Elements of a row laid out again: whole cache lines, so that a tile's pieces of
// a row meet no line of its neighbours.
int64_t pad(int64_t v) { return (v + 63) / 64 * 64; }
// Whether rows of v elements have to be laid out again: not whole 16-byte pieces.
bool odd_rows(int64_t v, int io) { return v % (io == SSD_BF16 ? 8 : 4) != 0; }
int64_t esz(int io) { return io == SSD_BF16 ? 2 : 4; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kCus = 256;       // compute units of the part this is written for
constexpr int64_t kFewRows = 32;    // rows that k_few can take
constexpr int64_t kFewOdd = 4;      // rows up to which it reads odd widths where they are

enum Tile { kT64, kT128, kT192, kTiles };
struct Shape {
    int bm, bn;
    int per_cu;        // workgroups a compute unit holds
    float alone, full; // us of a contraction step with one and with all of them (measured)
};
constexpr Shape kShape16[] = {{64, 64, 5, 0.42f, 0.90f}, {128, 128, 2, 0.85f, 1.0f},
                              {128, 192, 2, 0.83f, 1.13f}};
constexpr Shape kShape32[] = {{64, 64, 5, 0.70f, 2.6f}, {128, 128, 2, 3.0f, 3.9f}};

struct Product { int64_t m, n, k; };
struct Choice { Tile t; int64_t split[2]; };  // contraction parts of each product

// Time of a launch of products (us): rounds of workgroups times a step's time
// at the load of the last round; with several products, their work at full
// load and half a round's loss, but no less than the longest workgroup; and
// parts written and read back.  Over 33 products of 40 to 8192 rows timed in
// every tile and number of parts, what it chooses takes 1% more than the best of
// them on average, 7% at most.
float cost(const Shape &h, const Product *p, int count, const int64_t *split, int64_t bk) {
    int64_t all = 0, longest = 0;
    float work = 0.f, parts = 0.f;
    for (int i = 0; i < count; ++i) {
        const int64_t wgs = cdiv(p[i].m, h.bm) * cdiv(p[i].n, h.bn) * split[i];
        const int64_t steps = cdiv(cdiv(p[i].k, bk), split[i]);
        all += wgs;
        longest = steps > longest ? steps : longest;
        work += (float)wgs * steps;
        if (split[i] > 1) parts += 3.f + (float)split[i] * p[i].m * p[i].n * 8 / 4e6f;
    }
    const int64_t slots = kCus * h.per_cu, rounds = all / slots, rest = all % slots;
    const float load = (float)cdiv(rest, kCus);
    const float last = h.alone + (h.full - h.alone) * (load - 1) / (h.per_cu - 1);
    if (count == 1 || rounds == 0)
        return parts + longest * (rounds * h.full + (rest ? last : 0.f));
    return parts + work / slots * h.full + 0.5f * longest * h.full;
}

Choice choose(const Product *p, int count, int io) {
    constexpr int64_t kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
    const int64_t bk = 128 / esz(io);
    Choice best{kT128, {1, 1}};
    float least = 1e30f;
    for (int t = 0; t < (io == SSD_BF16 ? kTiles : 2); ++t)
        for (int64_t s0 : kSplits)
            for (int64_t s1 : kSplits) {
                const int64_t split[2] = {s0, s1};
                bool ok = count == 2 || s1 == 1;
                for (int i = 0; i < count; ++i)  // parts of four steps at least
                    ok = ok && (split[i] == 1 || cdiv(p[i].k, bk) / split[i] >= 4);
                if (!ok) continue;
                const float c = cost(io == SSD_BF16 ? kShape16[t] : kShape32[t], p, count, split, bk);
                if (c < least) least = c, best = {(Tile)t, {s0, s1}};
            }
    return best;
}

GemmArgs plan(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t m, int64_t n,
              int64_t k, const Choice &c, int which, const Epi &ep, float *parts, int io) {
    const Shape &h = io == SSD_BF16 ? kShape16[c.t] : kShape32[c.t];
    const int64_t bk = 128 / esz(io), steps = cdiv(k, bk);
    GemmArgs g{};
    g.A = A, g.B = B, g.lda = lda, g.ldb = ldb, g.m = m, g.n = n, g.k = k;
    g.tm = cdiv(m, h.bm), g.tn = cdiv(n, h.bn);
    g.kper = cdiv(steps, c.split[which]) * bk;
    g.split = cdiv(k, g.kper);
    g.parts = parts, g.ep = ep;
    return g;
}
size_t parts_bytes(const GemmArgs &g) {
    return g.split > 1 ? up((size_t)g.split * g.m * g.n * 4) : 0;
}

Choice choose_fwd(int64_t m, int64_t n, int64_t k, int io) {
    const Product p[1] = {{m, n, k}};
    return choose(p, 1, io);
}
Choice choose_bwd(int64_t m, int64_t n, int64_t k, int io) {
    const Product p[2] = {{m, k, n}, {n, k, m}};
    return choose(p, 2, io);
}

// Widths up to 2^20 elements, and tensors below 2^34 with their rows rounded up to
// 64: a tile's byte offsets stay below 2^30, pieces of four elements are counted
// in 32 bits, and so are the threads that lay two operands out again in one
// launch, a piece of eight each (the launch takes no more than 2^32).
bool linear_sizes(int64_t m, int64_t n, int64_t k) {
    const int64_t w = (int64_t)1 << 20, most = (int64_t)1 << 34;
    if (n > w || k > w || m >= ((int64_t)1 << 31)) return false;
    return m * pad(n) < most && m * pad(k) < most && n * pad(k) < most;
}

// Whether k_few takes a forward product of up to kFewRows rows, rather than the
// tiles.  A workgroup of it walks a whole contraction for 16 columns, with all rows
// of x for each: long contractions, and weights of more columns than one round of
// workgroups (256 x 16), take in proportion to their length and rows, more than
// 16 rows twice the matrix work; the tiles split a long contraction and read x
// once.  fp32 tiles are slower, and odd rows have to be laid out for them.  Of 732
// timed products of 1 to 32 rows this rule takes 0.5% (fp32 0.6%) more than the
// better of both on average, 28% at most, against 20% and three times with a
// rule on the rows alone.  bf16, k_few against tiles: 32 rows, 2560 -> 10576 23.1
// and 14.4 us, 16 rows 16.0 and 14.6, 5 rows 12.7 and 14.2; 32 rows, 768 -> 1536 5.0
// and 7.7; one row, 16384 -> 256 19.1 and 12.7.
bool few_fwd(int64_t m, int64_t n, int64_t k, int io) {
    if (m > kFewRows) return false;
    if (io == SSD_BF16) return k * (n > 4096 ? n : 4096) * (8 + (m > 16 ? 40 : m)) <= 600000000;
    if (odd_rows(k, io)) return true;
    return m <= 16 ? k <= 4096 || n > 2048 : k < 4096 && n * k <= ((int64_t)1 << 24);
}

// Whether a forward call lays its operands out again first.  k_few reads odd
// rows where they are; bf16 accesses off 4 bytes are slow enough that more than
// kFewOdd rows of x against a large weight repay the copies (2561 -> 10576, 16
// rows: 48 against 34 us; 333 -> 1000: 4.4 against 7.0).
bool pads(int64_t m, int64_t n, int64_t k, int io) {
    return odd_rows(k, io) &&
           (!few_fwd(m, n, k, io) || (io == SSD_BF16 && m > kFewOdd && n * k > (1 << 21)));
}

size_t fwd_bytes(int64_t m, int64_t n, int64_t k, int io) {
    const size_t copies = pads(m, n, k, io) ? up(m * pad(k) * esz(io)) + up(n * pad(k) * esz(io)) : 0;
    if (few_fwd(m, n, k, io)) return copies;
    return copies + parts_bytes(plan(nullptr, 0, nullptr, 0, m, n, k, choose_fwd(m, n, k, io), 0,
                                     Epi{}, nullptr, io));
}

template <typename IO>
int32_t run_linear(const void *x, const void *w, const Epi &ep, int64_t m, int64_t n, int64_t k,
                   char *ws, hipStream_t s) {
    const int io = sizeof(IO) == 2 ? SSD_BF16 : SSD_F32;
    int64_t ld = k;
    if (pads(m, n, k, io)) {
        PrepArgs p{};
        ld = pad(k);
        p.x = x, p.w = w, p.px = ws, p.pw = ws + up(m * ld * sizeof(IO));
        p.m = m, p.n = n, p.k = k, p.lk = ld;
        p.xb = cdiv(m * (ld / 8), 256), p.wb = cdiv(n * (ld / 8), 256);
        hipLaunchKernelGGL((k_pad<IO>), dim3((unsigned)(p.xb + p.wb)), dim3(256), 0, s, p);
        x = p.px, w = p.pw;
        ws = static_cast<char *>(p.pw) + up(n * ld * sizeof(IO));
    }
    if (few_fwd(m, n, k, io)) {
        GemmArgs g{};
        g.A = x, g.B = w, g.lda = g.ldb = ld, g.m = m, g.n = n, g.k = k, g.ep = ep;
        const dim3 grid((unsigned)cdiv(n, 16)), block(kFewWaves * 64);
        if (m <= 16)
            hipLaunchKernelGGL((k_few<IO, 1>), grid, block, 0, s, g);
        else
            hipLaunchKernelGGL((k_few<IO, 2>), grid, block, 0, s, g);
        return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
    }
    const Choice c = choose_fwd(m, n, k, io);
    const GemmArgs g = plan(x, ld, w, ld, m, n, k, c, 0, ep, reinterpret_cast<float *>(ws), io);
    const dim3 grid((unsigned)(g.tm * g.tn * g.split));
#define SSD_GEMM(BM, BN, WM, WN)                                                                  \
    hipLaunchKernelGGL((k_gemm<IO, BM, BN, WM, WN>), grid, dim3(WM * WN * 64), 0, s, g)
    if (c.t == kT64) SSD_GEMM(64, 64, 2, 2);
    else if (c.t == kT128) SSD_GEMM(128, 128, 2, 4);
    if constexpr (sizeof(IO) == 2)
        if (c.t == kT192) SSD_GEMM(128, 192, 2, 4);
#undef SSD_GEMM
    if (g.split > 1)
        hipLaunchKernelGGL((k_gemm_sum<IO>), dim3((unsigned)cdiv(m * cdiv(n, 4), 256)), dim3(256), 0,
                           s, g);
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

// Whether the gradient takes the one-pass kernel of few rows: for weights of 8 MB
// or more, where the bytes count (3 rows, 5712 x 4761 fp32: 53 against 110 us by
// the tiles); a smaller one is done sooner by the tiles (2 rows, 1000 x 1000
// bf16: 13 against 8 us).
bool few_bwd(int64_t m, int64_t n, int64_t k, int io) {
    return m <= kFewBwdRows && n * k * esz(io) >= (8 << 20);
}

// Parts of the gradient's workspace.
struct BwdWs {
    bool own_e;
    int64_t ln, lk, run, runs;
    Choice c;
    size_t e, w, x, part, px, pw, total;
    BwdWs(int64_t m, int64_t n, int64_t k, int act, int io) {
        const int64_t es = esz(io);
        if (few_bwd(m, n, k, io)) {
            // about four workgroups a compute unit, 64 to kFewRun weight rows each
            run = n * cdiv(k, 1024 / es) / (4 * kCus) / 16 * 16;
            run = run < 64 ? 64 : run > kFewRun ? kFewRun : run;
            runs = cdiv(n, run);
            px = 0, total = up(runs * m * k * 4);
            return;
        }
        own_e = act != SSD_ACT_NONE || odd_rows(n, io);
        ln = own_e ? pad(n) : n, lk = odd_rows(k, io) ? pad(k) : k;
        // 64 rows a workgroup, or 16 where that leaves compute units without one
        run = cdiv(m, 64) * cdiv(n, 512) >= 4 * kCus ? 64 : 16;
        runs = cdiv(m, run);
        c = choose_bwd(m, n, k, io);
        size_t o = 0;
        e = o, o += own_e ? up(m * ln * es) : 0;
        w = o, o += lk != k ? up(n * lk * es) : 0;
        x = o, o += lk != k ? up(m * lk * es) : 0;
        part = o, o += up(runs * n * 4);
        px = o, o += parts_bytes(plan(nullptr, 0, nullptr, 0, m, k, n, c, 0, Epi{}, nullptr, io));
        pw = o, o += parts_bytes(plan(nullptr, 0, nullptr, 0, n, k, m, c, 1, Epi{}, nullptr, io));
        total = o;
    }
};

template <typename IO>
int32_t run_few_bwd(const void *dy, const void *x, const void *w, const void *pre, int act, void *dx,
                    void *dw, float *db, int64_t m, int64_t n, int64_t k, const BwdWs &L, char *ws,
                    hipStream_t s) {
    PrepArgs p{};
    p.dy = dy, p.pre = act != SSD_ACT_NONE ? pre : nullptr, p.x = x, p.w = w, p.act = act;
    p.m = m, p.n = n, p.k = k, p.run = (int)L.run;
    GemmArgs gx{};
    gx.m = m, gx.n = k, gx.split = L.runs, gx.parts = reinterpret_cast<float *>(ws + L.px);
    gx.tm = dx != nullptr, gx.ep.out = dx;
    const dim3 grid((unsigned)(L.runs * cdiv(k, 1024 / (int64_t)sizeof(IO)))), block(256);
#define SSD_FEW(M)                                                                               \
    hipLaunchKernelGGL((k_few_bwd<IO, M>), grid, block, 0, s, p, gx, static_cast<IO *>(dw), db)
    if (m <= 1) SSD_FEW(1);
    else if (m <= 2) SSD_FEW(2);
    else if (m <= 4) SSD_FEW(4);
    else SSD_FEW(8);
#undef SSD_FEW
    if (dx)
        hipLaunchKernelGGL((k_few_sum<IO>), dim3((unsigned)cdiv(k, 128), (unsigned)m), dim3(256), 0, s,
                           gx);
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

template <typename IO>
int32_t run_linear_bwd(const void *dy, const void *x, const void *w, const void *pre, int act,
                       void *dx, void *dw, float *db, int64_t m, int64_t n, int64_t k, char *ws,
                       hipStream_t s) {
    const int io = sizeof(IO) == 2 ? SSD_BF16 : SSD_F32;
    const BwdWs L(m, n, k, act, io);
    if (few_bwd(m, n, k, io))
        return run_few_bwd<IO>(dy, x, w, pre, act, dx, dw, db, m, n, k, L, ws, s);
    PrepArgs p{};
    p.dy = dy, p.pre = act != SSD_ACT_NONE ? pre : nullptr, p.x = x, p.w = w, p.act = act;
    p.m = m, p.n = n, p.k = k, p.ln = L.ln, p.lk = L.lk, p.run = (int)L.run;
    if (L.own_e) p.e = ws + L.e;
    if (db) p.part = reinterpret_cast<float *>(ws + L.part);
    if (p.e || db) p.eb = L.runs * cdiv(L.ln, 512);
    if (L.lk != k && dw) p.px = ws + L.x, p.xb = cdiv(m * (L.lk / 8), 256);
    if (L.lk != k && dx) p.pw = ws + L.w, p.wb = cdiv(n * (L.lk / 8), 256);
    if (p.eb + p.xb + p.wb > 0)
        hipLaunchKernelGGL((k_bwd_prep<IO>), dim3((unsigned)(p.eb + p.xb + p.wb)), dim3(256), 0, s, p);
    const void *e = p.e ? p.e : dy;
    if (p.px) x = p.px;
    if (p.pw) w = p.pw;
    GemmArgs gx = plan(e, L.ln, w, L.lk, m, k, n, L.c, 0, Epi{dx, nullptr, nullptr, nullptr, 0},
                       reinterpret_cast<float *>(ws + L.px), io);
    GemmArgs gw = plan(e, L.ln, x, L.lk, n, k, m, L.c, 1, Epi{dw, nullptr, nullptr, nullptr, 0},
                       reinterpret_cast<float *>(ws + L.pw), io);
    if (!dx) gx.tm = 0;
    if (!dw) gw.tm = 0;
    const int64_t items = gx.tm * gx.tn * gx.split + gw.tm * gw.tn * gw.split;
    const int wfirst = gw.kper > gx.kper;
    if (items > 0) {
#define SSD_GEMM(BM, BN, WM, WN)                                                                  \
    hipLaunchKernelGGL((k_gemm_bwd<IO, BM, BN, WM, WN>), dim3((unsigned)items),               \
                       dim3(WM * WN * 64), 0, s, gx, gw, wfirst)
        if (L.c.t == kT64) SSD_GEMM(64, 64, 2, 2);
        else if (L.c.t == kT128) SSD_GEMM(128, 128, 2, 4);
        if constexpr (sizeof(IO) == 2)
            if (L.c.t == kT192) SSD_GEMM(128, 192, 2, 4);
#undef SSD_GEMM
    }
    const int64_t xb = dx && gx.split > 1 ? cdiv(m * cdiv(k, 4), 256) : 0;
    const int64_t wb = dw && gw.split > 1 ? cdiv(n * cdiv(k, 4), 256) : 0;
    const int64_t bb = db ? cdiv(n, 32) : 0;
    if (xb + wb + bb > 0)
        hipLaunchKernelGGL((k_bwd_finish<IO>), dim3((unsigned)(xb + wb + bb)), dim3(256), 0, s, gx, gw,
                           xb, wb, p.part, L.runs, db);
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

bool act_ok(int act) { return act >= SSD_ACT_NONE && act <= SSD_ACT_SIGMOID; }

}  // namespace

}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_linear_workspace_bytes(int64_t rows, int64_t in_dim, int64_t out_dim, int32_t io_dtype) {
    if ((io_dtype != SSD_F32 && io_dtype != SSD_BF16) || rows <= 0 || in_dim <= 0 || out_dim <= 0 ||
        !linear_sizes(rows, out_dim, in_dim))
        return 0;
    return fwd_bytes(rows, out_dim, in_dim, io_dtype);
}

size_t ssd_linear_bwd_workspace_bytes(int64_t rows, int64_t in_dim, int64_t out_dim,
                                      int32_t activation, int32_t io_dtype) {
    if ((io_dtype != SSD_F32 && io_dtype != SSD_BF16) || rows <= 0 || in_dim <= 0 || out_dim <= 0 ||
        !act_ok(activation) || !linear_sizes(rows, out_dim, in_dim))
        return 0;
    return BwdWs(rows, out_dim, in_dim, activation, io_dtype).total;
}

int32_t ssd_linear(const void *x, const void *weight, const float *bias, const void *residual,
                   void *out, void *pre, int32_t activation, int64_t rows, int64_t in_dim,
                   int64_t out_dim, int32_t io_dtype, void *workspace, size_t workspace_bytes,
                   void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || in_dim <= 0 || out_dim <= 0) return SSD_ERR_SHAPE;
    if (!act_ok(activation) || !linear_sizes(rows, out_dim, in_dim)) return SSD_ERR_UNSUPPORTED;
    if (rows == 0) return SSD_OK;
    if (!x || !weight || !out) return SSD_ERR_NULL;
    const int64_t es = esz(io_dtype);
    if (!row_al(x, in_dim, es) || !row_al(weight, in_dim, es) || !al(bias, 4) ||
        !row_al(residual, out_dim, es) || !row_al(out, out_dim, es) || !row_al(pre, out_dim, es))
        return SSD_ERR_ALIGN;
    const size_t need = ssd_linear_workspace_bytes(rows, in_dim, out_dim, io_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const Epi ep{out, bias, residual, pre, activation};
    char *ws = static_cast<char *>(workspace);
    return io_dtype == SSD_BF16 ? run_linear<bf16>(x, weight, ep, rows, out_dim, in_dim, ws, s)
                                : run_linear<float>(x, weight, ep, rows, out_dim, in_dim, ws, s);
}

int32_t ssd_linear_bwd(const void *dy, const void *x, const void *weight, const void *pre,
                       int32_t activation, void *dx, void *dweight, float *dbias, int64_t rows,
                       int64_t in_dim, int64_t out_dim, int32_t io_dtype, void *workspace,
                       size_t workspace_bytes, void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || in_dim <= 0 || out_dim <= 0) return SSD_ERR_SHAPE;
    if (!act_ok(activation) || !linear_sizes(rows, out_dim, in_dim))
        return SSD_ERR_UNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int64_t es = esz(io_dtype);
    if (!row_al(dx, in_dim, es) || !row_al(dweight, in_dim, es) || !al(dbias, 4))
        return SSD_ERR_ALIGN;
    if (rows == 0) {
        // no rows: the weight's and the bias's gradients are zero
        const int64_t n = out_dim * in_dim;
        const unsigned blocks = (unsigned)(cdiv(n, 256) < 65536 ? cdiv(n, 256) : 65536);
        if (dweight && io_dtype == SSD_BF16)
            hipLaunchKernelGGL((k_zero<bf16>), dim3(blocks), dim3(256), 0, s, static_cast<bf16 *>(dweight), n);
        else if (dweight)
            hipLaunchKernelGGL((k_zero<float>), dim3(blocks), dim3(256), 0, s, static_cast<float *>(dweight), n);
        if (dbias)
            hipLaunchKernelGGL((k_zero<float>), dim3((unsigned)((out_dim + 255) / 256)), dim3(256), 0,
                               s, dbias, out_dim);
        return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
    }
    if (!dy || (dx && !weight) || (dweight && !x) || (activation != SSD_ACT_NONE && !pre))
        return SSD_ERR_NULL;
    if (!row_al(dy, out_dim, es) || !row_al(x, in_dim, es) || !row_al(weight, in_dim, es) ||
        !row_al(pre, out_dim, es))
        return SSD_ERR_ALIGN;
    const size_t need = BwdWs(rows, out_dim, in_dim, activation, io_dtype).total;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    char *ws = static_cast<char *>(workspace);
    return io_dtype == SSD_BF16
               ? run_linear_bwd<bf16>(dy, x, weight, pre, activation, dx, dweight, dbias, rows,
                                      out_dim, in_dim, ws, s)
               : run_linear_bwd<float>(dy, x, weight, pre, activation, dx, dweight, dbias, rows,
                                       out_dim, in_dim, ws, s);
}

}  // extern "C"
