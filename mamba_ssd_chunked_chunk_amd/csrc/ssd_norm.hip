// Layer norm over the last axis, with the residual in front of it, and its
// gradient.  For a row s = x (+ residual, rounded to the io type):
//
//   mean = sum s / dim,  rstd = 1 / sqrt(sum (s - mean)^2 / dim + eps)
//   hat = (s - mean) rstd,  y = hat weight + bias
//   g = dy weight,  ds = rstd (g - mean(g) - hat mean(g hat)) (+ d_sum)
//   dweight = sum over rows of dy hat,  dbias = sum over rows of dy
//
// Bound by memory.  A row is read once and stays in the registers of the G
// lanes that own it (E elements each) until its outputs are written, so both
// passes over it (mean, then the squares about it, which do not cancel, and what is
// left of the mean) cost no traffic.  G is 8 or 32 lanes for short rows, a wave up to 4096 elements, a
// workgroup up to 16384; longer rows are read again for each pass.  All sums
// are fp32.  16384 rows of 2560 with residual and statistics, bf16: 66 us, 5.1 TB/s;
// their gradient 88 us, 3.8 TB/s, at two workgroups a compute unit (its registers
// are the column sums; the next row loaded ahead gave 85 us for 50 more of them).
//
// In the gradient a lane keeps the same columns for every row of its
// workgroup, so the column sums stay in registers too; each workgroup writes
// one row of partial sums, which a second kernel adds in order (the number of
// workgroups depends on the sizes alone, so results repeat bit for bit).
#include <hip/hip_runtime.h>

#include <math.h>
#include <initializer_list>

#include "../../include/ssd.h"
#include "ssd_device.hpp"

namespace ssd {

namespace {

constexpr int kNormThreads = 256;
constexpr int kMostLane = 64;                          // elements of a row per lane
constexpr int kMostRow = kNormThreads * kMostLane;     // longest row in registers
constexpr int kMostBlocks = 1024;                      // workgroups of the gradient, at most

template <typename IO, int V>
struct alignas(sizeof(IO) * V < 16 ? sizeof(IO) * V : 16) NVec { IO e[V]; };

struct NormArgs {
    const void *x, *r;          // forward: input and residual
    const float *weight, *bias;
    const void *dy, *dsum;      // gradient
    void *y, *sum;              // y or dx, x + residual
    const float *stats_in;
    float *stats;               // [2, rows] mean, rstd
    float *dw, *db;             // column sums (of workgroup 0; the others at `stride` floats)
    int64_t rows, dim, stride;
    float eps;
};

// Sum over the G lanes of a row; for G = 256 through LDS, where the two halves
// of `red` alternate so that one barrier per sum is enough.
template <int G> __device__ __forceinline__ float row_sum(float v, float *red, int &half) {
#pragma unroll
    for (int o = 1; o < (G < 64 ? G : 64); o <<= 1) v += __shfl_xor(v, o);
    if constexpr (G > 64) {
        float *p = red + 4 * half;
        half ^= 1;
        if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (p[0] + p[1]) + (p[2] + p[3]);
    }
    return v;
}

// 1 / deviation from the mean square about a value that the mean is u above.
__device__ __forceinline__ float norm_rstd(float sq, float u, float eps) {
    const float v = fmaf(-u, u, sq);
    return 1.f / sqrtf((v < 0.f ? 0.f : v) + eps);  // NaN stays NaN
}

template <typename IO, int V, int G, int E>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm(NormArgs a) {
    typedef NVec<IO, V> Vec;
    constexpr int K = E / V, RPB = kNormThreads / G;
    __shared__ float red[8];
    int half = 0;
    const int lane = threadIdx.x % G;
    const int nv = (int)(a.dim / V);
    const float inv = 1.f / (float)a.dim;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / G; row < a.rows;
         row += (int64_t)gridDim.x * RPB) {
        const Vec *px = reinterpret_cast<const Vec *>(static_cast<const IO *>(a.x) + row * a.dim);
        float s[E];
        Vec xv[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) xv[k] = px[k * G + lane];
        if (a.r) {
            const Vec *pr = reinterpret_cast<const Vec *>(static_cast<const IO *>(a.r) + row * a.dim);
            Vec rv[K];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k * G + lane < nv) rv[k] = pr[k * G + lane];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k * G + lane < nv) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        xv[k].e[e] = (IO)(to_f32(xv[k].e[e]) + to_f32(rv[k].e[e]));
                    if (a.sum)
                        reinterpret_cast<Vec *>(static_cast<IO *>(a.sum) + row * a.dim)[k * G + lane] =
                            xv[k];
                }
        }
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = k * G + lane < nv;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[k * V + e] = in ? to_f32(xv[k].e[e]) : 0.f;
                t += s[k * V + e];
            }
        }
        // The mean of a row far from zero is off by roundings of it that can be more than
        // the row deviates by: what is left of the mean after it is taken off (the
        // difference is then exact, or nearly so) is taken off too, and from the squares.
        const float mean = row_sum<G>(t, red, half) * inv;
        float u = 0.f;
        t = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[k * V + e] -= mean;
                    u += s[k * V + e];
                    t = fmaf(s[k * V + e], s[k * V + e], t);
                }
            }
        u = row_sum<G>(u, red, half) * inv;
        const float rstd = norm_rstd(row_sum<G>(t, red, half) * inv, u, a.eps);
        if (a.stats && lane == 0) a.stats[row] = mean + u, a.stats[a.rows + row] = rstd;
        Vec *py = reinterpret_cast<Vec *>(static_cast<IO *>(a.y) + row * a.dim);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) {
                const int c = k * G + lane;
                NVec<float, V> w, b;
#pragma unroll
                for (int e = 0; e < V; ++e) w.e[e] = 1.f, b.e[e] = 0.f;
                if (a.weight) w = reinterpret_cast<const NVec<float, V> *>(a.weight)[c];
                if (a.bias) b = reinterpret_cast<const NVec<float, V> *>(a.bias)[c];
                Vec o;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o.e[e] = (IO)fmaf((s[k * V + e] - u) * rstd, w.e[e], b.e[e]);
                py[c] = o;
            }
    }
}

template <typename IO, int V, int G, int E>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_bwd(NormArgs a) {
    typedef NVec<IO, V> Vec;
    constexpr int K = E / V, RPB = kNormThreads / G;
    extern __shared__ float cols[];  // [2][dim] (G <= 64)
    __shared__ float red[8];
    int half = 0;
    const int lane = threadIdx.x % G;
    const int nv = (int)(a.dim / V);
    const float inv = 1.f / (float)a.dim;
    float sw[E], sb[E];
#pragma unroll
    for (int i = 0; i < E; ++i) sw[i] = sb[i] = 0.f;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / G; row < a.rows;
         row += (int64_t)gridDim.x * RPB) {
        const int64_t at = row * a.dim;
        const Vec *px = reinterpret_cast<const Vec *>(static_cast<const IO *>(a.x) + at);
        const Vec *pd = reinterpret_cast<const Vec *>(static_cast<const IO *>(a.dy) + at);
        // the row's values as they were read; widened where they are used
        Vec xv[K], dv[K], more[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) xv[k] = px[k * G + lane], dv[k] = pd[k * G + lane];
        if (a.dsum) {
            const Vec *ps = reinterpret_cast<const Vec *>(static_cast<const IO *>(a.dsum) + at);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k * G + lane < nv) more[k] = ps[k * G + lane];
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) more[k].e[e] = (IO)0.f;
        }
        const float mean = a.stats_in[row], rstd = a.stats_in[a.rows + row];
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) {
                NVec<float, V> w;
#pragma unroll
                for (int e = 0; e < V; ++e) w.e[e] = 1.f;
                if (a.weight) w = reinterpret_cast<const NVec<float, V> *>(a.weight)[k * G + lane];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = to_f32(dv[k].e[e]), hat = (to_f32(xv[k].e[e]) - mean) * rstd;
                    const float g = d * w.e[e];
                    c1 += g;
                    c2 = fmaf(g, hat, c2);
                    sw[k * V + e] = fmaf(d, hat, sw[k * V + e]);
                    sb[k * V + e] += d;
                }
            }
        if (!a.y) continue;
        c1 = row_sum<G>(c1, red, half) * inv;
        c2 = row_sum<G>(c2, red, half) * inv;
        Vec *po = reinterpret_cast<Vec *>(static_cast<IO *>(a.y) + at);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) {
                const int c = k * G + lane;
                NVec<float, V> w;
                Vec o;
#pragma unroll
                for (int e = 0; e < V; ++e) w.e[e] = 1.f;
                if (a.weight) w = reinterpret_cast<const NVec<float, V> *>(a.weight)[c];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float hat = (to_f32(xv[k].e[e]) - mean) * rstd;
                    const float g = to_f32(dv[k].e[e]) * w.e[e];
                    o.e[e] = (IO)fmaf(rstd, g - c1 - hat * c2, to_f32(more[k].e[e]));
                }
                po[c] = o;
            }
    }
    if (!a.dw && !a.db) return;
    // rows of one wave that share a column, then the waves in order
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int o = G; o < 64; o <<= 1) {
            sw[i] += __shfl_xor(sw[i], o);
            sb[i] += __shfl_xor(sb[i], o);
        }
    float *dw = a.dw ? a.dw + blockIdx.x * a.stride : nullptr;
    float *db = a.db ? a.db + blockIdx.x * a.stride : nullptr;
    if constexpr (G <= 64) {
        const int wave = threadIdx.x >> 6;
        for (int w = 0; w < kNormThreads / 64; ++w) {
            if (wave == w && (threadIdx.x & 63) < G) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k * G + lane < nv) {
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const int c = (k * G + lane) * V + e;
                            cols[c] = w ? cols[c] + sw[k * V + e] : sw[k * V + e];
                            cols[a.dim + c] = w ? cols[a.dim + c] + sb[k * V + e] : sb[k * V + e];
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < (int)a.dim; c += kNormThreads) {
            if (dw) dw[c] = cols[c];
            if (db) db[c] = cols[a.dim + c];
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * G + lane < nv) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int c = (k * G + lane) * V + e;
                    if (dw) dw[c] = sw[k * V + e];
                    if (db) db[c] = sb[k * V + e];
                }
            }
    }
}

// Rows beyond the registers: a workgroup reads its row again for each pass.
template <typename IO>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_wide(NormArgs a) {
    __shared__ float red[8];
    int half = 0;
    const float inv = 1.f / (float)a.dim;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const IO *px = static_cast<const IO *>(a.x) + row * a.dim;
        const IO *pr = a.r ? static_cast<const IO *>(a.r) + row * a.dim : nullptr;
        IO *psum = a.sum && pr ? static_cast<IO *>(a.sum) + row * a.dim : nullptr;
        IO *py = static_cast<IO *>(a.y) + row * a.dim;
        // `first`: the sum is formed and written; later passes read it back
        // (each element by the thread that wrote it), so that it may be x
        const auto value = [&](int64_t c, bool first) {
            if (!pr || (psum && !first)) return to_f32(psum && pr ? psum[c] : px[c]);
            const IO v = (IO)(to_f32(px[c]) + to_f32(pr[c]));
            if (psum) psum[c] = v;
            return to_f32(v);
        };
        float t = 0.f;
        for (int64_t c = threadIdx.x; c < a.dim; c += kNormThreads) t += value(c, true);
        const float mean = row_sum<kNormThreads>(t, red, half) * inv;
        float u = 0.f;
        t = 0.f;
        for (int64_t c = threadIdx.x; c < a.dim; c += kNormThreads) {
            const float d = value(c, false) - mean;
            u += d;
            t = fmaf(d, d, t);
        }
        u = row_sum<kNormThreads>(u, red, half) * inv;
        const float rstd = norm_rstd(row_sum<kNormThreads>(t, red, half) * inv, u, a.eps);
        if (a.stats && threadIdx.x == 0) a.stats[row] = mean + u, a.stats[a.rows + row] = rstd;
        for (int64_t c = threadIdx.x; c < a.dim; c += kNormThreads)
            py[c] = (IO)fmaf((value(c, false) - mean - u) * rstd, a.weight ? a.weight[c] : 1.f,
                             a.bias ? a.bias[c] : 0.f);
    }
}

template <typename IO>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_bwd_wide(NormArgs a) {
    __shared__ float red[8];
    int half = 0;
    const float inv = 1.f / (float)a.dim;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const IO *px = static_cast<const IO *>(a.x) + row * a.dim;
        const IO *pd = static_cast<const IO *>(a.dy) + row * a.dim;
        const IO *ps = a.dsum ? static_cast<const IO *>(a.dsum) + row * a.dim : nullptr;
        IO *po = static_cast<IO *>(a.y) + row * a.dim;
        const float mean = a.stats_in[row], rstd = a.stats_in[a.rows + row];
        float c1 = 0.f, c2 = 0.f;
        for (int64_t c = threadIdx.x; c < a.dim; c += kNormThreads) {
            const float g = to_f32(pd[c]) * (a.weight ? a.weight[c] : 1.f);
            c1 += g;
            c2 = fmaf(g, (to_f32(px[c]) - mean) * rstd, c2);
        }
        c1 = row_sum<kNormThreads>(c1, red, half) * inv;
        c2 = row_sum<kNormThreads>(c2, red, half) * inv;
        for (int64_t c = threadIdx.x; c < a.dim; c += kNormThreads) {
            const float g = to_f32(pd[c]) * (a.weight ? a.weight[c] : 1.f);
            const float hat = (to_f32(px[c]) - mean) * rstd;
            po[c] = (IO)fmaf(rstd, g - c1 - hat * c2, ps ? to_f32(ps[c]) : 0.f);
        }
    }
}

// Column sums of long rows: a thread per column, rows in strips over blockIdx.y.
template <typename IO>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_cols(NormArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= a.dim) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float d = to_f32(static_cast<const IO *>(a.dy)[row * a.dim + c]);
        const float v = to_f32(static_cast<const IO *>(a.x)[row * a.dim + c]);
        sw = fmaf(d, (v - a.stats_in[row]) * a.stats_in[a.rows + row], sw);
        sb += d;
    }
    if (a.dw) a.dw[blockIdx.y * a.stride + c] = sw;
    if (a.db) a.db[blockIdx.y * a.stride + c] = sb;
}

// The workgroups' partial sums [blocks][2 dim]: V columns a thread, added in order
// by 32 strips whose sums are added in order.
template <int V>
__global__ __launch_bounds__(256) void k_layer_norm_sum(const float *__restrict__ part, float *dw,
                                                        float *db, int blocks, int64_t dim) {
    typedef NVec<float, V> Vec;
    __shared__ Vec red[32][8];
    const int col = threadIdx.x & 7, strip = threadIdx.x >> 3;
    const int64_t c = ((int64_t)blockIdx.x * 8 + col) * V;
    Vec t;
#pragma unroll
    for (int e = 0; e < V; ++e) t.e[e] = 0.f;
    if (c < 2 * dim) {
#pragma unroll 8
        for (int b = strip; b < blocks; b += 32) {
            const Vec v = *reinterpret_cast<const Vec *>(part + (int64_t)b * 2 * dim + c);
#pragma unroll
            for (int e = 0; e < V; ++e) t.e[e] += v.e[e];
        }
    }
    red[strip][col] = t;
    __syncthreads();
    if (strip == 0 && c < 2 * dim) {
#pragma unroll
        for (int i = 1; i < 32; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) t.e[e] += red[i][col].e[e];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (c + e < dim) {
                if (dw) dw[c + e] = t.e[e];
            } else if (db) {
                db[c + e - dim] = t.e[e];
            }
        }
    }
}

__global__ void k_layer_norm_zero(float *dw, float *db, int64_t dim) {
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < dim;
         c += (int64_t)gridDim.x * 256) {
        if (dw) dw[c] = 0.f;
        if (db) db[c] = 0.f;
    }
}

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Elements that move at once: 16 bytes of the io type where every row and
// every tensor allow it, else 2 bf16 elements, else one.
template <typename IO> int norm_vec(int64_t dim, const float *f0, const float *f1,
                                    std::initializer_list<const void *> io) {
    for (int v : {(int)(16 / sizeof(IO)), 2}) {
        if (sizeof(IO) == 4 && v == 2) break;
        bool ok = dim % v == 0 && al(f0, v >= 4 ? 16 : 4 * v) && al(f1, v >= 4 ? 16 : 4 * v);
        for (const void *p : io) ok = ok && al(p, v * sizeof(IO));
        if (ok) return v;
    }
    return 1;
}

// Lanes of a row and elements per lane: the fewest lanes that hold it eight
// elements each (so short rows share a wave), else a wave, else a workgroup.
struct NormShape {
    int g, e;
    explicit NormShape(int64_t dim) {
        if (dim <= 64) g = 8, e = 8;
        else if (dim <= 256) g = 32, e = 8;
        else if (dim <= 64 * kMostLane) {
            g = 64;
            const int per = (int)((dim + 63) / 64);
            e = per <= 8 ? 8 : per <= 16 ? 16 : per <= 24 ? 24 : per <= 32 ? 32 : per <= 40 ? 40
                : per <= 48 ? 48 : 64;
        } else {
            g = kNormThreads;
            e = dim <= kNormThreads * 32 ? 32 : 64;
        }
    }
    int rows_per_block() const { return kNormThreads / g; }
};

template <typename IO, int V, int G, int E>
hipError_t norm_go(const NormArgs &a, bool bwd, int blocks, hipStream_t s) {
    if (bwd)
        hipLaunchKernelGGL((k_layer_norm_bwd<IO, V, G, E>), dim3(blocks), dim3(kNormThreads),
                           G <= 64 && (a.dw || a.db) ? 2 * a.dim * 4 : 0, s, a);
    else
        hipLaunchKernelGGL((k_layer_norm<IO, V, G, E>), dim3(blocks), dim3(kNormThreads), 0, s, a);
    return hipGetLastError();
}

template <typename IO, int V>
hipError_t norm_shape(const NormArgs &a, bool bwd, const NormShape &n, int blocks, hipStream_t s) {
    if (n.g == 8) return norm_go<IO, V, 8, 8>(a, bwd, blocks, s);
    if (n.g == 32) return norm_go<IO, V, 32, 8>(a, bwd, blocks, s);
    if (n.g == kNormThreads)
        return n.e == 32 ? norm_go<IO, V, kNormThreads, 32>(a, bwd, blocks, s)
                         : norm_go<IO, V, kNormThreads, 64>(a, bwd, blocks, s);
    switch (n.e) {
    case 8: return norm_go<IO, V, 64, 8>(a, bwd, blocks, s);
    case 16: return norm_go<IO, V, 64, 16>(a, bwd, blocks, s);
    case 24: return norm_go<IO, V, 64, 24>(a, bwd, blocks, s);
    case 32: return norm_go<IO, V, 64, 32>(a, bwd, blocks, s);
    case 40: return norm_go<IO, V, 64, 40>(a, bwd, blocks, s);
    case 48: return norm_go<IO, V, 64, 48>(a, bwd, blocks, s);
    default: return norm_go<IO, V, 64, 64>(a, bwd, blocks, s);
    }
}

template <typename IO>
hipError_t norm_vecs(const NormArgs &a, bool bwd, int v, const NormShape &n, int blocks,
                     hipStream_t s) {
    if (v == (int)(16 / sizeof(IO))) return norm_shape<IO, 16 / sizeof(IO)>(a, bwd, n, blocks, s);
    if constexpr (sizeof(IO) == 2)
        if (v == 2) return norm_shape<IO, 2>(a, bwd, n, blocks, s);
    return norm_shape<IO, 1>(a, bwd, n, blocks, s);
}

bool norm_sizes(int64_t rows, int64_t dim) {
    return dim <= ((int64_t)1 << 24) && rows <= ((int64_t)1 << 40) / dim;
}

// Workgroups of the gradient: four on a compute unit where a lane has 16 columns or
// fewer, else two.  Two do run at once up to 48 columns a lane with bf16 io and 40 with
// fp32, up to 32 where elements move one at a time; above that, and where 256 lanes
// have a row whose elements do, the registers of the column sums leave room for one.
// 16384 rows of 2560 take 93 us in 512 workgroups, 114 in 768 or 1024.  Fewer rows than
// that go one to each of G lanes, though a row of partial sums is then written for few
// of them: 1999 rows of 771 take 20 us so, 27 us with four rows to each.
int norm_blocks(int64_t rows, int64_t dim) {
    const NormShape n(dim);
    const int64_t slots = n.e <= 16 ? kMostBlocks : kMostBlocks / 2;
    const int64_t b = (rows + n.rows_per_block() - 1) / n.rows_per_block();
    // beyond 16 MB of partial sums (rows wider than 4096) fewer workgroups run: 198 of
    // them, less than one a compute unit, for rows of 10576
    const int64_t most = ((int64_t)1 << 24) / (8 * dim);
    const int64_t cap = most < 1 ? 1 : most > slots ? slots : most;
    return (int)(b < cap ? b : cap);
}

template <typename IO> hipError_t norm_fwd(const NormArgs &a, hipStream_t s) {
    if (a.dim > kMostRow) {
        const int64_t b = a.rows < 65536 ? a.rows : 65536;
        hipLaunchKernelGGL(k_layer_norm_wide<IO>, dim3((unsigned)b), dim3(kNormThreads), 0, s, a);
        return hipGetLastError();
    }
    const NormShape n(a.dim);
    const int rpb = n.rows_per_block();
    int64_t b = (a.rows + rpb - 1) / rpb;
    if (b > 65536) b = 65536;
    const int v = norm_vec<IO>(a.dim, a.weight, a.bias, {a.x, a.r, a.y, a.sum});
    return norm_vecs<IO>(a, false, v, n, (int)b, s);
}

template <typename IO>
hipError_t norm_bwd(NormArgs a, float *dw, float *db, float *part, hipStream_t s) {
    const int blocks = norm_blocks(a.rows, a.dim);
    const bool sums = dw || db;
    a.dw = a.db = nullptr;
    if (sums && blocks == 1) {
        a.dw = dw, a.db = db;
    } else if (sums) {
        a.dw = part, a.db = part + a.dim, a.stride = 2 * a.dim;
    }
    hipError_t e = hipSuccess;
    if (a.dim > kMostRow) {
        if (sums) {
            hipLaunchKernelGGL(k_layer_norm_cols<IO>,
                               dim3((unsigned)((a.dim + kNormThreads - 1) / kNormThreads), blocks),
                               dim3(kNormThreads), 0, s, a);
            e = hipGetLastError();
        }
        if (a.y && e == hipSuccess) {
            const int64_t b = a.rows < 65536 ? a.rows : 65536;
            hipLaunchKernelGGL(k_layer_norm_bwd_wide<IO>, dim3((unsigned)b), dim3(kNormThreads), 0, s,
                               a);
            e = hipGetLastError();
        }
    } else {
        const int v = norm_vec<IO>(a.dim, a.weight, nullptr, {a.x, a.dy, a.y, a.dsum});
        e = norm_vecs<IO>(a, true, v, NormShape(a.dim), blocks, s);
    }
    if (sums && blocks > 1 && e == hipSuccess) {
        const int64_t per = a.dim % 2 ? 16 : 32;  // columns of a workgroup
        const dim3 grid((unsigned)((2 * a.dim + per - 1) / per));
        hipLaunchKernelGGL(a.dim % 2 ? &k_layer_norm_sum<2> : &k_layer_norm_sum<4>, grid, dim3(256), 0,
                           s, part, dw, db, blocks, a.dim);
        e = hipGetLastError();
    }
    return e;
}

bool io_al(int io, std::initializer_list<const void *> p) {
    for (const void *q : p)
        if (!al(q, io == SSD_BF16 ? 2 : 4)) return false;
    return true;
}

}  // namespace

}  // namespace ssd

using namespace ssd;

extern "C" {

int32_t ssd_layer_norm(const void *x, const void *residual, const float *weight, const float *bias,
                       float eps, void *y, void *sum, float *stats, int64_t rows, int64_t dim,
                       int32_t io_dtype, void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || dim <= 0 || !(eps >= 0.f)) return SSD_ERR_SHAPE;
    if (!norm_sizes(rows, dim)) return SSD_ERR_UNSUPPORTED;
    if (rows == 0) return SSD_OK;
    if (!x || !y || (sum && !residual)) return SSD_ERR_NULL;
    if (!io_al(io_dtype, {x, residual, y, sum}) || !al(weight, 4) || !al(bias, 4) || !al(stats, 4))
        return SSD_ERR_ALIGN;
    NormArgs a{};
    a.x = x, a.r = residual, a.weight = weight, a.bias = bias, a.eps = eps, a.y = y, a.sum = sum;
    a.stats = stats, a.rows = rows, a.dim = dim;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const hipError_t e = io_dtype == SSD_BF16 ? norm_fwd<bf16>(a, s) : norm_fwd<float>(a, s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

size_t ssd_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
    if (rows <= 0 || dim <= 0 || !norm_sizes(rows, dim)) return 0;
    const int blocks = norm_blocks(rows, dim);
    return blocks == 1 ? 0 : (size_t)blocks * 2 * dim * 4;
}

int32_t ssd_layer_norm_bwd(const void *dy, const void *x, const float *stats, const float *weight,
                           const void *d_sum, void *dx, float *dweight, float *dbias, int64_t rows,
                           int64_t dim, int32_t io_dtype, void *workspace, size_t workspace_bytes,
                           void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (rows < 0 || dim <= 0) return SSD_ERR_SHAPE;
    if (!norm_sizes(rows, dim)) return SSD_ERR_UNSUPPORTED;
    if (!dx && !dweight && !dbias) return SSD_ERR_NULL;
    if (!al(dweight, 4) || !al(dbias, 4)) return SSD_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (rows == 0) {
        if (!dweight && !dbias) return SSD_OK;
        int64_t b = (dim + 255) / 256;
        if (b > 4096) b = 4096;
        hipLaunchKernelGGL(k_layer_norm_zero, dim3((unsigned)b), dim3(256), 0, s, dweight, dbias, dim);
        return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
    }
    if (!dy || !x || !stats) return SSD_ERR_NULL;
    if (!io_al(io_dtype, {dy, x, d_sum, dx}) || !al(stats, 4) || !al(weight, 4)) return SSD_ERR_ALIGN;
    const size_t need =
        dweight || dbias ? ssd_layer_norm_bwd_workspace_bytes(rows, dim) : 0;
    if (need && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (need && !al(workspace, 256)) return SSD_ERR_ALIGN;
    NormArgs a{};
    a.dy = dy, a.x = x, a.stats_in = stats, a.weight = weight, a.dsum = d_sum, a.y = dx;
    a.rows = rows, a.dim = dim;
    float *part = static_cast<float *>(workspace);
    const hipError_t e = io_dtype == SSD_BF16 ? norm_bwd<bf16>(a, dweight, dbias, part, s)
                                              : norm_bwd<float>(a, dweight, dbias, part, s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // extern "C"
