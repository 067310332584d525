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

#include "../../include/ssd.h"
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
__device__ __forceinline__ float act_f(float v, int act) {
    if (act == SSD_ACT_SILU) return v * __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
    if (act == SSD_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.7071067811865476f));
    if (act == SSD_ACT_SIGMOID) return __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
    return v;
}
__device__ __forceinline__ float act_grad(float v, int act) {
    if (act == SSD_ACT_GELU)
        return 0.5f * (1.f + erff(v * 0.7071067811865476f)) +
               0.3989422804014327f * v * exp2_fast(-0.5f * kLog2e * v * v);
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
    void *out;           // io elements, or fp32 parts [split][m][n]
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
    Epi ep;
};

// Four consecutive n of one row m.
template <typename IO>
__device__ __forceinline__ void finish4(const Epi &ep, int64_t m, int64_t n, int64_t N, f32x4 v) {
    const int64_t at = m * N + n;
    if (n + 4 <= N && N % 4 == 0) {
        if (ep.bias) {
            f32x4 b;
            __builtin_memcpy(&b, ep.bias + n, 16);
            v += b;
        }
        if (ep.pre) st4<IO>(static_cast<IO *>(ep.pre) + at, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_f(v[i], ep.act);
        if (ep.res) v += ld4<IO>(static_cast<const IO *>(ep.res) + at);
        st4<IO>(static_cast<IO *>(ep.out) + at, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= N) break;
        float x = v[i];
        if (ep.bias) x += ep.bias[n + i];
        if (ep.pre) static_cast<IO *>(ep.pre)[at + i] = (IO)x;
        x = act_f(x, ep.act);
        if (ep.res) x += to_f32(static_cast<const IO *>(ep.res)[at + i]);
        static_cast<IO *>(ep.out)[at + i] = (IO)x;
    }
}

// ------------------------------------------------------------ LDS tiles ----
// An operand's tile is ROWS stored rows of 16-byte chunks, CH chunks a row,
// chunk c of row r kept at slot c ^ f(r).
//   contraction contiguous: ROWS = tile rows m, a row is 128 bytes of k
//   contraction outermost:  ROWS = 128 / sizeof(IO) values of k, a row is the tile's m
template <typename IO, bool TR, int BM> struct OpTile {
    static constexpr int EPC = 16 / (int)sizeof(IO);
    static constexpr int BK = 128 / (int)sizeof(IO);
    static constexpr int ROWS = TR ? BK : BM;
    static constexpr int CH = TR ? BM / EPC : 8;
    static constexpr int BYTES = ROWS * CH * 16;
    static __device__ __forceinline__ int f(int r) {
        if (!TR) return r & 7;
        if (sizeof(IO) == 2) return (((r & 3) | ((r >> 1) & 4)) << 1) & (CH - 1);
        return (((r >> 2) & 3) << 2) & (CH - 1);
    }
};

template <typename IO, bool TR, int BM, int NT>
__device__ __forceinline__ void stage(const GemmArgs &g, const void *src, int64_t ld, int64_t m0,
                                      int64_t mEnd, int64_t k0, int64_t kEnd, char *lds) {
    typedef OpTile<IO, TR, BM> T;
    const int tid = threadIdx.x;
    const IO *base;
    int64_t bytes;
    if (TR) {
        base = static_cast<const IO *>(src) + k0 * ld + m0;
        bytes = ((kEnd - k0) * ld - m0) * (int64_t)sizeof(IO);
    } else {
        base = static_cast<const IO *>(src) + m0 * ld + k0;
        bytes = ((mEnd - m0) * ld - k0) * (int64_t)sizeof(IO);
    }
    // offsets inside a tile stay below 2^31, so a resource never has to reach
    // further, and the offset of a masked piece lies past every resource
    const RsrcW r = make_rsrc_w(base, bytes < 0x7fffffff ? bytes : 0x7fffffff);
    constexpr int N = T::BYTES / 16 / NT;
    static_assert(T::BYTES % (16 * NT) == 0, "tile copies");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int slot = i * NT + tid, row = slot / T::CH, ch = (slot % T::CH) ^ T::f(row);
        uint32_t off = (uint32_t)(row * ld + ch * T::EPC) * (uint32_t)sizeof(IO);
        if (!TR && k0 + ch * T::EPC >= kEnd) off = 0xffffff00u;
        lds_dma16(r, (lds_void *)(lds + (i * NT + (tid & ~63)) * 16), off);
    }
}

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

// One workgroup: a BM x BN tile of D over one contraction part.  WM x WN waves.
template <typename IO, bool TA, bool TB, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void k_gemm(GemmArgs g) {
    constexpr int NT = WM * WN * 64;
    typedef OpTile<IO, TA, BM> OA;
    typedef OpTile<IO, TB, BN> OB;
    constexpr int BK = OA::BK;
    constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    __shared__ __align__(16) char lds[2][OA::BYTES + OB::BYTES];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int64_t part = item / (g.tm * g.tn), tile = item % (g.tm * g.tn);
    const int64_t m0 = tile / g.tn * BM, n0 = tile % g.tn * BN;
    const int64_t k0 = part * g.kper, kEnd = k0 + g.kper < g.k ? k0 + g.kper : g.k;
    const int wm = wv / WN * (BM / WM), wn = wv % WN * (BN / WN);
    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = zero4();
    auto copy = [&](int64_t k, int buf) {
        stage<IO, TA, BM, NT>(g, g.A, g.lda, m0, g.m, k, kEnd, lds[buf]);
        stage<IO, TB, BN, NT>(g, g.B, g.ldb, n0, g.n, k, kEnd, lds[buf] + OA::BYTES);
    };
    int buf = 0;
    copy(k0, 0);
    for (int64_t k = k0; k < kEnd; k += BK) {
        vm_wait<0>();
        lds_barrier();
        if (k + BK < kEnd) copy(k + BK, buf ^ 1);
        const char *a = lds[buf], *b = lds[buf] + OA::BYTES;
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
        buf ^= 1;
    }
    // element r of a lane: row m of lane & 15, column 4 (lane >> 4) + r
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + wm + 16 * i + (lane & 15);
        if (m >= g.m) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t n = n0 + wn + 16 * j + 4 * (lane >> 4);
            if (n >= g.n) continue;
            if (g.split > 1) {
                float *p = static_cast<float *>(g.ep.out) + (part * g.m + m) * g.n + n;
                if (g.n % 4 == 0)
                    *reinterpret_cast<f32x4 *>(p) = acc[i][j];
                else
                    for (int r = 0; r < 4 && n + r < g.n; ++r) p[r] = acc[i][j][r];
            } else {
                finish4<IO>(g.ep, m, n, g.n, acc[i][j]);
            }
        }
    }
}

// Sums the contraction parts in order and finishes the elements.
template <typename IO>
__global__ __launch_bounds__(256) void k_gemm_sum(const float *parts, int64_t split, int64_t m,
                                                  int64_t n, Epi ep) {
    const int64_t q = (n + 3) / 4, k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= m * q) return;
    const int64_t row = k / q, col = k % q * 4;
    f32x4 v = zero4();
    for (int64_t s = 0; s < split; ++s) {
        const float *p = parts + (s * m + row) * n + col;
        if (n % 4 == 0)
            v += *reinterpret_cast<const f32x4 *>(p);
        else
            for (int r = 0; r < 4 && col + r < n; ++r) v[r] += p[r];
    }
    finish4<IO>(ep, row, col, n, v);
}

// --------------------------------------------------------------- helpers ----
// Rows of `cols` elements laid out again with `ld` elements a row, zeros behind them.
template <typename IO>
__global__ __launch_bounds__(256) void k_pad_rows(const IO *src, IO *dst, int64_t rows, int64_t cols,
                                                  int64_t ld) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        if (c < ld) dst[r * ld + c] = c < cols ? src[r * cols + c] : (IO)0.f;
}

// e = dy act'(pre) in the io type (e NULL: not written) with ld elements a row
// and zeros behind the row, and its fp32 sums over runs of kBiasRows rows.
constexpr int kBiasRows = 64;
template <typename IO>
__global__ __launch_bounds__(256) void k_act_bwd(const IO *dy, const IO *pre, IO *e, float *part,
                                                 int64_t m, int64_t n, int64_t ld, int act) {
    const int64_t c = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (c >= ld) return;
    const int64_t r0 = (int64_t)blockIdx.x * kBiasRows;
    const int64_t r1 = r0 + kBiasRows < m ? r0 + kBiasRows : m;
    float s = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        float v = 0.f;
        if (c < n) {
            v = to_f32(dy[r * n + c]);
            if (pre) v *= act_grad(to_f32(pre[r * n + c]), act);
        }
        s += v;
        if (e) e[r * ld + c] = (IO)v;
    }
    if (part && c < n) part[blockIdx.x * n + c] = s;
}

__global__ __launch_bounds__(256) void k_bias_sum(const float *part, float *db, int64_t rows,
                                                  int64_t n) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float s = 0.f;
    for (int64_t r = 0; r < rows; ++r) s += part[r * n + c];
    db[c] = s;
}

template <typename IO>
__global__ __launch_bounds__(256) void k_zero(IO *p, int64_t n) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k < n) p[k] = (IO)0.f;
}

// --------------------------------------------------------------- the plan ----
size_t up(size_t v) { return (v + 255) & ~(size_t)255; }
int64_t pad(int64_t v, int io) { return io == SSD_BF16 ? (v + 7) / 8 * 8 : (v + 3) / 4 * 4; }
int64_t esz(int io) { return io == SSD_BF16 ? 2 : 4; }

constexpr int kBM = 128, kBN = 128;

// Contraction parts of a product: as many as it takes to give every compute
// unit a workgroup, none shorter than 8 steps.
int64_t parts_of(int64_t m, int64_t n, int64_t k, int io) {
    const int64_t tiles = (m + kBM - 1) / kBM * ((n + kBN - 1) / kBN), step = 128 / esz(io);
    const int64_t steps = (k + step - 1) / step;
    int64_t s = 256 / tiles;
    if (s > steps / 8) s = steps / 8;
    return s < 1 ? 1 : s;
}
size_t parts_bytes(int64_t m, int64_t n, int64_t k, int io) {
    const int64_t s = parts_of(m, n, k, io);
    return s > 1 ? up((size_t)s * m * n * 4) : 0;
}

template <typename IO, bool TA, bool TB>
hipError_t product(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t m, int64_t n,
                   int64_t k, const Epi &ep, float *parts, hipStream_t s) {
    const int io = sizeof(IO) == 2 ? SSD_BF16 : SSD_F32;
    const int64_t step = 128 / (int64_t)sizeof(IO), steps = (k + step - 1) / step;
    GemmArgs g{};
    g.A = A, g.B = B, g.lda = lda, g.ldb = ldb, g.m = m, g.n = n, g.k = k;
    g.tm = (m + kBM - 1) / kBM, g.tn = (n + kBN - 1) / kBN;
    g.split = parts_of(m, n, k, io);
    g.kper = (steps + g.split - 1) / g.split * step;
    g.split = (k + g.kper - 1) / g.kper;
    g.ep = ep;
    if (g.split > 1) g.ep.out = parts;
    hipLaunchKernelGGL((k_gemm<IO, TA, TB, kBM, kBN, 2, 2>), dim3((unsigned)(g.tm * g.tn * g.split)),
                       dim3(256), 0, s, g);
    if (g.split > 1)
        hipLaunchKernelGGL((k_gemm_sum<IO>), dim3((unsigned)((m * ((n + 3) / 4) + 255) / 256)),
                           dim3(256), 0, s, parts, g.split, m, n, ep);
    return hipGetLastError();
}

template <typename IO>
void pad_rows(const void *src, void *dst, int64_t rows, int64_t cols, int64_t ld, hipStream_t s) {
    const int64_t y = rows < 4096 ? rows : 4096;
    hipLaunchKernelGGL((k_pad_rows<IO>), dim3((unsigned)((ld + 255) / 256), (unsigned)y), dim3(256), 0,
                       s, static_cast<const IO *>(src), static_cast<IO *>(dst), rows, cols, ld);
}

// Widths up to 2^20 elements and rows up to 2^31: a tile's byte offsets stay
// below 2^31 and every grid below 2^31 workgroups.
bool linear_sizes(int64_t m, int64_t n, int64_t k) {
    const int64_t w = (int64_t)1 << 20;
    if (n > w || k > w || m >= ((int64_t)1 << 31)) return false;
    const int64_t big = ((int64_t)1 << 31) - 1;
    return (m + 127) / 128 * ((n + 127) / 128) <= big && m * ((n + 3) / 4) / 256 < big;
}

template <typename IO>
int32_t run_linear(const void *x, const void *w, const Epi &ep, int64_t m, int64_t n, int64_t k,
                   char *ws, hipStream_t s) {
    const int io = sizeof(IO) == 2 ? SSD_BF16 : SSD_F32;
    const int64_t ld = pad(k, io);
    if (ld != k) {
        char *px = ws, *pw = ws + up(m * ld * sizeof(IO));
        pad_rows<IO>(x, px, m, k, ld, s);
        pad_rows<IO>(w, pw, n, k, ld, s);
        x = px, w = pw;
        ws = pw + up(n * ld * sizeof(IO));
    }
    const hipError_t e = product<IO, false, false>(x, ld, w, ld, m, n, k, ep,
                                                   reinterpret_cast<float *>(ws), s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

// Parts of the gradient's workspace.
struct BwdWs {
    size_t e, w, x, part, prod, total;
    BwdWs(int64_t m, int64_t n, int64_t k, int act, int io) {
        const int64_t ln = pad(n, io), lk = pad(k, io), es = esz(io);
        size_t o = 0;
        e = o, o += act != SSD_ACT_NONE || ln != n ? up(m * ln * es) : 0;
        w = o, o += lk != k ? up(n * lk * es) : 0;
        x = o, o += lk != k ? up(m * lk * es) : 0;
        part = o, o += up((m + kBiasRows - 1) / kBiasRows * n * 4);
        const size_t p1 = parts_bytes(m, k, n, io), p2 = parts_bytes(n, k, m, io);
        prod = o, o += p1 > p2 ? p1 : p2;
        total = o;
    }
};

template <typename IO>
int32_t run_linear_bwd(const void *dy, const void *x, const void *w, const void *pre, int act,
                       void *dx, void *dw, float *db, int64_t m, int64_t n, int64_t k, char *ws,
                       hipStream_t s) {
    const int io = sizeof(IO) == 2 ? SSD_BF16 : SSD_F32;
    const int64_t ln = pad(n, io), lk = pad(k, io);
    const BwdWs L(m, n, k, act, io);
    const bool own_e = act != SSD_ACT_NONE || ln != n;
    const void *e = own_e ? ws + L.e : dy;
    if (own_e || db) {
        const int64_t rows = (m + kBiasRows - 1) / kBiasRows;
        hipLaunchKernelGGL((k_act_bwd<IO>), dim3((unsigned)rows, (unsigned)((ln + 255) / 256)),
                           dim3(256), 0, s, static_cast<const IO *>(dy),
                           static_cast<const IO *>(act != SSD_ACT_NONE ? pre : nullptr),
                           own_e ? reinterpret_cast<IO *>(ws + L.e) : nullptr,
                           db ? reinterpret_cast<float *>(ws + L.part) : nullptr, m, n, ln, act);
        if (db)
            hipLaunchKernelGGL(k_bias_sum, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                               reinterpret_cast<const float *>(ws + L.part), db, rows, n);
    }
    if (lk != k) {
        if (dx) pad_rows<IO>(w, ws + L.w, n, k, lk, s);
        if (dw) pad_rows<IO>(x, ws + L.x, m, k, lk, s);
        w = ws + L.w, x = ws + L.x;
    }
    float *parts = reinterpret_cast<float *>(ws + L.prod);
    hipError_t r = hipGetLastError();
    Epi ep{};
    if (dx && r == hipSuccess) {
        ep.out = dx;
        r = product<IO, false, true>(e, ln, w, lk, m, k, n, ep, parts, s);
    }
    if (dw && r == hipSuccess) {
        ep.out = dw;
        r = product<IO, true, true>(e, ln, x, lk, n, k, m, ep, parts, s);
    }
    return r == hipSuccess ? SSD_OK : SSD_ERR_HIP;
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
    const int64_t ld = pad(in_dim, io_dtype), es = esz(io_dtype);
    const size_t copies = ld != in_dim ? up(rows * ld * es) + up(out_dim * ld * es) : 0;
    return copies + parts_bytes(rows, out_dim, in_dim, io_dtype);
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
    if (!act_ok(activation) || !linear_sizes(rows, out_dim, in_dim) ||
        !linear_sizes(out_dim, in_dim, 1))
        return SSD_ERR_UNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int64_t es = esz(io_dtype);
    if (!row_al(dx, in_dim, es) || !row_al(dweight, in_dim, es) || !al(dbias, 4))
        return SSD_ERR_ALIGN;
    if (rows == 0) {
        // no rows: the weight's and the bias's gradients are zero
        const int64_t n = out_dim * in_dim;
        if (dweight && io_dtype == SSD_BF16)
            hipLaunchKernelGGL((k_zero<bf16>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                               static_cast<bf16 *>(dweight), n);
        else if (dweight)
            hipLaunchKernelGGL((k_zero<float>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                               static_cast<float *>(dweight), n);
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
