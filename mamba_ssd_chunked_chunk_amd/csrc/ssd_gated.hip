// The gated linear recurrence, per channel c of x [b, l, d]:
//
//   u_t = scale softplus(lam_c) sigmoid(r_t)     a_t = e^{-u_t}
//   h_t = a_t h_{t-1} + v_t,  v_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t,  y_t = h_t
//
// with r_t = gates[.., c] and i_t = gates[.., d + c] raw (before their
// sigmoids), its gradient, and one decode step of it.
//
// A tile is T = kSeg * NW tokens of 64 * V channels: a lane owns V channels,
// a wave a run of kSeg consecutive tokens, so every load of a wave is one
// contiguous piece of a token's row.  A run is the map h -> A h + S of the
// state entering it (A = prod a_t, S its result from zero); runs compose in
// order: waves through LDS inside a tile, tiles through the workspace.
#include <hip/hip_runtime.h>

#include <math.h>

#include "../../include/ssd.h"
#include "ssd_device.hpp"

namespace ssd {

namespace {

constexpr int kSeg = 8;    // tokens per wave
constexpr int kGW = 8;     // waves per workgroup
constexpr int kGT = kSeg * kGW;  // tokens per tile
static_assert(kGT % SSD_GATED_CHUNK == 0 && SSD_GATED_CHUNK % kSeg == 0, "tile and state spacing");
constexpr float kLn2 = 0.6931471805599453f;

template <typename IO, int V> struct alignas(sizeof(IO) * V) VecIO { IO e[V]; };
template <int V> struct alignas(4 * V) VecF { float e[V]; };

__device__ __forceinline__ float sigmoid_f(float z) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(-z * kLog2e));
}

// softplus(v) = max(v, 0) + log1p(e^-|v|)
__device__ __forceinline__ float softplus_f(float v) {
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

// a = e^-u and beta = sqrt(1 - a^2) for u = u2 ln 2 >= 0.  1 - a^2 =
// -expm1(-2u) is taken from its series where the subtraction would cancel:
// t = 2u < 1/4, six terms, relative error t^6 / 5040 < 2^-24; above, the
// subtraction loses at most two bits of fp32.
__device__ __forceinline__ void decay(float u2, float &a, float &beta) {
    a = exp2_fast(-u2);
    const float t = 2.f * kLn2 * u2;
    const float s =
        t * (1.f - t * (0.5f - t * (1.f / 6 - t * (1.f / 24 - t * (1.f / 120 - t * (1.f / 720))))));
    beta = __builtin_amdgcn_sqrtf(t < 0.25f ? s : 1.f - a * a);
}

struct GArgs {
    const void *x, *gates;
    const float *lam;
    float scale;
    const float *init;
    const int32_t *seq;
    const float *kept;    // backward: states after every SSD_GATED_CHUNK tokens
    const void *dy;       // backward
    const float *dfin;    // backward
    void *y;              // forward output, or dx
    void *dgates;
    float *fin;           // final state, or d_init
    float *states;        // forward output: states after every SSD_GATED_CHUNK tokens
    float *part;          // backward: per tile sums behind dlam [b, tiles, d]
    float *A, *S, *R;     // workspace: per tile maps [b, tiles, d]
    int64_t b, l, d, tiles;
};

// What one tile's loads need: this lane's channels and its rows.
template <typename IO, int V> struct Tile {
    int64_t c;       // first channel of this lane (clamped to a valid one)
    bool live;       // the lane's channels exist
    int64_t row0;    // the sequence's first row in [b * l]
    int64_t t0;      // the wave's first token
    __device__ Tile(const GArgs &g, int64_t bi, int64_t tile) {
        const int lane = threadIdx.x & 63;
        c = ((int64_t)blockIdx.x * 64 + lane) * V;
        live = c < g.d;
        if (!live) c = 0;
        row0 = bi * g.l;
        t0 = tile * kGT + wave_id() * kSeg;
    }
};

template <typename IO, int V>
__device__ __forceinline__ VecIO<IO, V> ldv(const void *p, int64_t at) {
    return *reinterpret_cast<const VecIO<IO, V> *>(static_cast<const IO *>(p) + at);
}
template <typename IO, int V>
__device__ __forceinline__ void stv(void *p, int64_t at, const VecIO<IO, V> &v) {
    *reinterpret_cast<VecIO<IO, V> *>(static_cast<IO *>(p) + at) = v;
}

// The wave's rows of x, r and i (rows past the end read the last row).
template <typename IO, int V> struct Rows {
    VecIO<IO, V> x[kSeg], r[kSeg], i[kSeg];
    __device__ void load(const GArgs &g, const Tile<IO, V> &w) {
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            int64_t t = w.t0 + k;
            if (t >= g.l) t = g.l - 1;
            const int64_t at = (w.row0 + t) * g.d + w.c;
            x[k] = ldv<IO, V>(g.x, at);
            r[k] = ldv<IO, V>(g.gates, at + (w.row0 + t) * g.d);
            i[k] = ldv<IO, V>(g.gates, at + (w.row0 + t + 1) * g.d);
        }
    }
};

// Whether token t takes the state of the token before it (the first token
// takes the initial state).
__device__ __forceinline__ bool same_document(const GArgs &g, int64_t row0, int64_t t) {
    if (!g.seq || t <= 0 || t >= g.l) return true;
    return g.seq[row0 + t] == g.seq[row0 + t - 1];
}

// Decay and added value of the wave's tokens; identity past the end.
template <typename IO, int V>
__device__ __forceinline__ void terms(const GArgs &g, const Tile<IO, V> &w, const Rows<IO, V> &rw,
                                      const float (&m2)[V], float (&a)[kSeg][V],
                                      float (&v)[kSeg][V]) {
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        const int64_t t = w.t0 + k;
        const bool in = t < g.l, same = same_document(g, w.row0, t);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float aa, beta;
            decay(m2[e] * sigmoid_f(to_f32(rw.r[k].e[e])), aa, beta);
            const float vv = beta * sigmoid_f(to_f32(rw.i[k].e[e])) * to_f32(rw.x[k].e[e]);
            a[k][e] = in ? (same ? aa : 0.f) : 1.f;
            v[k][e] = in ? vv : 0.f;
        }
    }
}

template <typename IO, int V>
__device__ __forceinline__ void rates(const GArgs &g, const Tile<IO, V> &w, float (&m2)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) m2[e] = g.scale * softplus_f(g.lam[w.c + e]) * kLog2e;
}

// ------------------------------------------------------------- forward ----
// Every tile's map (A, S), and for the backward pass the adjoint's R.
template <typename IO, int V, bool FWD, bool ADJ>
__global__ __launch_bounds__(kGW * 64, 2) void k_gated_map(GArgs g) {
    __shared__ VecF<V> sA[kGW][64], sS[kGW][64], sR[kGW][64];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int64_t tile = blockIdx.y, bi = blockIdx.z;
    const Tile<IO, V> w(g, bi, tile);
    float m2[V];
    rates(g, w, m2);
    Rows<IO, V> rw;
    rw.load(g, w);
    float a[kSeg][V], v[kSeg][V];
    terms(g, w, rw, m2, a, v);
    VecF<V> A, S, R;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float p = 1.f, s = 0.f;
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            p *= a[k][e];
            s = a[k][e] * s + v[k][e];
        }
        A.e[e] = p;
        S.e[e] = s;
    }
    if constexpr (ADJ) {
#pragma unroll
        for (int e = 0; e < V; ++e) R.e[e] = 0.f;
#pragma unroll
        for (int k = kSeg - 1; k >= 0; --k) {
            const int64_t t = w.t0 + k;
            const VecIO<IO, V> dy = ldv<IO, V>(
                g.dy, (w.row0 + (t < g.l ? t : g.l - 1)) * g.d + w.c);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (t < g.l) R.e[e] = a[k][e] * (to_f32(dy.e[e]) + R.e[e]);
        }
        sR[wv][lane] = R;
    }
    sA[wv][lane] = A;
    sS[wv][lane] = S;
    __syncthreads();
    if (wv != 0 || !w.live) return;
    VecF<V> tA, tS, tR;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float p = 1.f, s = 0.f, q = 0.f;
#pragma unroll
        for (int j = 0; j < kGW; ++j) {
            p *= sA[j][lane].e[e];
            s = sA[j][lane].e[e] * s + sS[j][lane].e[e];
        }
        if constexpr (ADJ) {
#pragma unroll
            for (int j = kGW - 1; j >= 0; --j) q = sA[j][lane].e[e] * q + sR[j][lane].e[e];
        }
        tA.e[e] = p;
        tS.e[e] = s;
        tR.e[e] = q;
    }
    const int64_t at = (bi * g.tiles + tile) * g.d + w.c;
    *reinterpret_cast<VecF<V> *>(g.A + at) = tA;
    if constexpr (FWD) *reinterpret_cast<VecF<V> *>(g.S + at) = tS;
    if constexpr (ADJ) *reinterpret_cast<VecF<V> *>(g.R + at) = tR;
}

// Turns every tile's S into the state entering it and (backward) every
// tile's R into the adjoint carry entering it from its right.
template <bool FWD, bool ADJ>
__global__ __launch_bounds__(256) void k_gated_chain(GArgs g) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= g.b * g.d) return;
    const int64_t bi = k / g.d, c = k % g.d, base = bi * g.tiles * g.d + c;
    if constexpr (FWD) {
        float h = g.init ? g.init[k] : 0.f;
        for (int64_t j = 0; j < g.tiles; ++j) {
            const float A = g.A[base + j * g.d], S = g.S[base + j * g.d];
            g.S[base + j * g.d] = h;
            h = A * h + S;
        }
    }
    if constexpr (ADJ) {
        float q = g.dfin ? g.dfin[k] : 0.f;
        for (int64_t j = g.tiles - 1; j >= 0; --j) {
            const float A = g.A[base + j * g.d], R = g.R[base + j * g.d];
            g.R[base + j * g.d] = q;
            q = A * q + R;
        }
    }
}

// The states of a tile's tokens from the state entering it.
template <typename IO, int V>
__global__ __launch_bounds__(kGW * 64, 2) void k_gated_out(GArgs g) {
    __shared__ VecF<V> sA[kGW][64], sS[kGW][64];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int64_t tile = blockIdx.y, bi = blockIdx.z;
    const Tile<IO, V> w(g, bi, tile);
    float m2[V];
    rates(g, w, m2);
    Rows<IO, V> rw;
    rw.load(g, w);
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        h[e] = g.tiles > 1 ? g.S[(bi * g.tiles + tile) * g.d + w.c + e]
                           : (g.init ? g.init[bi * g.d + w.c + e] : 0.f);
    float a[kSeg][V], v[kSeg][V];
    terms(g, w, rw, m2, a, v);
    VecF<V> A, S;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float p = 1.f, s = 0.f;
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            p *= a[k][e];
            s = a[k][e] * s + v[k][e];
        }
        A.e[e] = p;
        S.e[e] = s;
    }
    sA[wv][lane] = A;
    sS[wv][lane] = S;
    __syncthreads();
    if (w.t0 >= g.l) return;
#pragma unroll
    for (int j = 0; j < kGW - 1; ++j)
        if (j < wv) {
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] = sA[j][lane].e[e] * h[e] + sS[j][lane].e[e];
        }
    if (!w.live) return;
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        const int64_t t = w.t0 + k;
        VecIO<IO, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            h[e] = a[k][e] * h[e] + v[k][e];
            o.e[e] = (IO)h[e];
        }
        if (t < g.l) stv<IO, V>(g.y, (w.row0 + t) * g.d + w.c, o);
    }
    const int64_t end = w.t0 + kSeg < g.l ? w.t0 + kSeg : g.l;
    VecF<V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.e[e] = h[e];
    if (g.states && (end == g.l || end % SSD_GATED_CHUNK == 0)) {
        const int64_t ns = (g.l + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK;
        *reinterpret_cast<VecF<V> *>(
            g.states + (bi * ns + (end - 1) / SSD_GATED_CHUNK) * g.d + w.c) = o;
    }
    if (g.fin && end == g.l) *reinterpret_cast<VecF<V> *>(g.fin + bi * g.d + w.c) = o;
}

// ------------------------------------------------------------ backward ----
// g_t = dy_t + q_t, q_{t-1} = a_t g_t (q entering the sequence from its right
// is d_final, q_{-1} the gradient of the initial state); then
//   dx = g beta sigmoid(i),  di = g beta x sigmoid(i) (1 - sigmoid(i)),
//   p  = u dL/du = g (a^2 (u / beta) sigmoid(i) x - u a h_{t-1}),
//   dr = p (1 - sigmoid(r)),  dlam = sum p sigmoid(lam) / softplus(lam).
// u / beta = u / sqrt(1 - e^{-2u}) goes to zero with u, so nothing divides by
// zero where the decay rounds to one.
template <typename IO, int V>
__global__ __launch_bounds__(kGW * 64, 2) void k_gated_bwd(GArgs g) {
    __shared__ VecF<V> sA[kGW][64], sS[kGW][64], sR[kGW][64];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int64_t tile = blockIdx.y, bi = blockIdx.z;
    const Tile<IO, V> w(g, bi, tile);
    float m2[V];
    rates(g, w, m2);
    Rows<IO, V> rw;
    rw.load(g, w);
    VecIO<IO, V> dy[kSeg];
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        const int64_t t = w.t0 + k < g.l ? w.t0 + k : g.l - 1;
        dy[k] = ldv<IO, V>(g.dy, (w.row0 + t) * g.d + w.c);
    }
    float h[V], q[V];
    const int64_t ns = (g.l + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int64_t ch = w.c + e, at = (bi * g.tiles + tile) * g.d + ch;
        if (tile == 0)
            h[e] = g.init ? g.init[bi * g.d + ch] : 0.f;
        else if (g.kept)
            h[e] = g.kept[(bi * ns + tile * kGT / SSD_GATED_CHUNK - 1) * g.d + ch];
        else
            h[e] = g.S[at];
        q[e] = tile < g.tiles - 1 ? g.R[at] : (g.dfin ? g.dfin[bi * g.d + ch] : 0.f);
    }
    float a[kSeg][V], v[kSeg][V];
    terms(g, w, rw, m2, a, v);
    VecF<V> A, S, R;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float p = 1.f, s = 0.f, r = 0.f;
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            p *= a[k][e];
            s = a[k][e] * s + v[k][e];
        }
#pragma unroll
        for (int k = kSeg - 1; k >= 0; --k)
            if (w.t0 + k < g.l) r = a[k][e] * (to_f32(dy[k].e[e]) + r);
        A.e[e] = p;
        S.e[e] = s;
        R.e[e] = r;
    }
    sA[wv][lane] = A;
    sS[wv][lane] = S;
    sR[wv][lane] = R;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kGW; ++j)
        if (j < wv) {
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] = sA[j][lane].e[e] * h[e] + sS[j][lane].e[e];
        }
#pragma unroll
    for (int j = kGW - 1; j >= 0; --j)
        if (j > wv) {
#pragma unroll
            for (int e = 0; e < V; ++e) q[e] = sA[j][lane].e[e] * q[e] + sR[j][lane].e[e];
        }
    __syncthreads();
    // the states before every token, in place of the added values
#pragma unroll
    for (int k = 0; k < kSeg; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float hn = a[k][e] * h[e] + v[k][e];
            v[k][e] = h[e];
            h[e] = hn;
        }
    VecF<V> acc;
#pragma unroll
    for (int e = 0; e < V; ++e) acc.e[e] = 0.f;
#pragma unroll
    for (int k = kSeg - 1; k >= 0; --k) {
        const int64_t t = w.t0 + k;
        if (t >= g.l) continue;
        VecIO<IO, V> ox, orr, oi;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float gt = to_f32(dy[k].e[e]) + q[e];
            const float sr = sigmoid_f(to_f32(rw.r[k].e[e])), si = sigmoid_f(to_f32(rw.i[k].e[e]));
            const float x = to_f32(rw.x[k].e[e]), u2 = m2[e] * sr, u = kLn2 * u2;
            float aa, beta;
            decay(u2, aa, beta);
            const float ratio = beta > 0.f ? u * __builtin_amdgcn_rcpf(beta) : 0.f;
            const float gx = gt * si;
            const float p = aa * aa * ratio * gx * x - u * a[k][e] * gt * v[k][e];
            ox.e[e] = (IO)(gx * beta);
            oi.e[e] = (IO)(gx * beta * x * (1.f - si));
            orr.e[e] = (IO)(p * (1.f - sr));
            acc.e[e] += p;
            q[e] = a[k][e] * gt;
        }
        if (w.live) {
            const int64_t at = (w.row0 + t) * g.d + w.c;
            stv<IO, V>(g.y, at, ox);
            stv<IO, V>(g.dgates, at + (w.row0 + t) * g.d, orr);
            stv<IO, V>(g.dgates, at + (w.row0 + t + 1) * g.d, oi);
        }
    }
    sS[wv][lane] = acc;
    __syncthreads();
    if (wv != 0 || !w.live) return;
    VecF<V> s;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s.e[e] = 0.f;
#pragma unroll
        for (int j = 0; j < kGW; ++j) s.e[e] += sS[j][lane].e[e];
    }
    *reinterpret_cast<VecF<V> *>(g.part + (bi * g.tiles + tile) * g.d + w.c) = s;
    if (g.fin && tile == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) s.e[e] = q[e];
        *reinterpret_cast<VecF<V> *>(g.fin + bi * g.d + w.c) = s;
    }
}

// dlam: the tiles' sums, added in a fixed order in fp64.  One workgroup: 32
// channels by 8 runs of tiles.
__global__ __launch_bounds__(256) void k_gated_lam(const float *part, const float *lam, float *dlam,
                                                   int64_t rows, int64_t d) {
    __shared__ double s[8][32];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t ch = (int64_t)blockIdx.x * 32 + c;
    double t = 0;
    if (ch < d)
        for (int64_t j = k; j < rows; j += 8) t += part[j * d + ch];
    s[k][c] = t;
    __syncthreads();
    if (k != 0 || ch >= d) return;
#pragma unroll
    for (int j = 1; j < 8; ++j) t += s[j][c];
    // sigmoid(v) / softplus(v) tends to one as v goes to minus infinity
    const double v = lam[ch];
    const double ratio = v < -30. ? 1. : 1. / ((1. + exp(-v)) * (fmax(v, 0.) + log1p(exp(-fabs(v)))));
    dlam[ch] = (float)(t * ratio);
}

// ---------------------------------------------------------------- step ----
template <typename IO, int V>
__global__ __launch_bounds__(256) void k_gated_step(float *state, const IO *x, const IO *gates,
                                                    const float *lam, float scale, IO *y,
                                                    int64_t b, int64_t d) {
    const int64_t n = b * (d / V);
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= n) return;
    const int64_t bi = k / (d / V), c = (k % (d / V)) * V, at = bi * d + c;
    VecF<V> h = *reinterpret_cast<const VecF<V> *>(state + at);
    const VecF<V> lm = *reinterpret_cast<const VecF<V> *>(lam + c);
    const VecIO<IO, V> xv = ldv<IO, V>(x, at), r = ldv<IO, V>(gates, at + bi * d),
                       i = ldv<IO, V>(gates, at + (bi + 1) * d);
    VecIO<IO, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float a, beta;
        decay(scale * softplus_f(lm.e[e]) * kLog2e * sigmoid_f(to_f32(r.e[e])), a, beta);
        h.e[e] = a * h.e[e] + beta * sigmoid_f(to_f32(i.e[e])) * to_f32(xv.e[e]);
        o.e[e] = (IO)h.e[e];
    }
    *reinterpret_cast<VecF<V> *>(state + at) = h;
    stv<IO, V>(y, at, o);
}

// batch > 0, seqlen == 0: the final state is the initial one, or zeros
__global__ void k_gated_copy(float *dst, const float *src, int64_t n) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k < n) dst[k] = src ? src[k] : 0.f;
}

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Workspace: A, S (the backward pass also R and the sums behind dlam), each
// [b, tiles, d] fp32.
size_t gated_ws(int64_t b, int64_t l, int64_t d, int parts) {
    const int64_t tiles = (l + kGT - 1) / kGT;
    const size_t one = ((size_t)b * tiles * d * 4 + 255) & ~(size_t)255;
    return parts * one;
}

// Channels a lane moves at once: 4 or 2 where the width and every tensor allow
// vector accesses of as many elements, else 1.
template <typename... P> int lanes(int io, int64_t d, const float *f0, const float *f1,
                                   P... p) {
    for (int v = 4; v > 1; v /= 2) {
        const uintptr_t a = v * (io == SSD_BF16 ? 2 : 4), f = 4 * v;
        if (d % v == 0 && al(f0, f) && al(f1, f) && (al(p, a) && ...))
            return v;
    }
    return 1;
}
template <typename... P> bool io_aligned(int io, P... p) {
    return (al(p, io == SSD_BF16 ? 2 : 4) && ...);
}

// sizes whose element offsets and grids fit
bool gated_sizes(int64_t b, int64_t l, int64_t d) {
    return b <= 65535 && d <= ((int64_t)1 << 24) && l <= (int64_t)65535 * kGT;
}

template <typename IO, int V> hipError_t fwd(GArgs &g, hipStream_t s) {
    const dim3 grid((unsigned)((g.d + 64 * V - 1) / (64 * V)), (unsigned)g.tiles, (unsigned)g.b);
    if (g.tiles > 1) {
        hipLaunchKernelGGL((k_gated_map<IO, V, true, false>), grid, dim3(kGW * 64), 0, s, g);
        hipLaunchKernelGGL((k_gated_chain<true, false>),
                           dim3((unsigned)((g.b * g.d + 255) / 256)), dim3(256), 0, s, g);
    }
    hipLaunchKernelGGL((k_gated_out<IO, V>), grid, dim3(kGW * 64), 0, s, g);
    return hipGetLastError();
}

template <typename IO, int V> hipError_t bwd(GArgs &g, float *dlam, hipStream_t s) {
    const dim3 grid((unsigned)((g.d + 64 * V - 1) / (64 * V)), (unsigned)g.tiles, (unsigned)g.b);
    const dim3 line((unsigned)((g.b * g.d + 255) / 256));
    if (g.tiles > 1) {
        if (g.kept) {
            hipLaunchKernelGGL((k_gated_map<IO, V, false, true>), grid, dim3(kGW * 64), 0, s, g);
            hipLaunchKernelGGL((k_gated_chain<false, true>), line, dim3(256), 0, s, g);
        } else {
            hipLaunchKernelGGL((k_gated_map<IO, V, true, true>), grid, dim3(kGW * 64), 0, s, g);
            hipLaunchKernelGGL((k_gated_chain<true, true>), line, dim3(256), 0, s, g);
        }
    }
    hipLaunchKernelGGL((k_gated_bwd<IO, V>), grid, dim3(kGW * 64), 0, s, g);
    hipLaunchKernelGGL(k_gated_lam, dim3((unsigned)((g.d + 31) / 32)), dim3(256), 0, s, g.part,
                       g.lam, dlam, g.b * g.tiles, g.d);
    return hipGetLastError();
}

}  // namespace

}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_gated_scan_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
    if (batch <= 0 || seqlen <= 0 || dim <= 0 || !gated_sizes(batch, seqlen, dim)) return 0;
    return gated_ws(batch, seqlen, dim, 2);
}

size_t ssd_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
    if (batch <= 0 || seqlen <= 0 || dim <= 0 || !gated_sizes(batch, seqlen, dim)) return 0;
    return gated_ws(batch, seqlen, dim, 4);
}

int32_t ssd_gated_scan(const void *x, const void *gates, const float *lam, float scale,
                       const float *init_state, const int32_t *seq_idx, void *y,
                       float *final_state, float *states, int64_t batch, int64_t seqlen,
                       int64_t dim, int32_t io_dtype, void *workspace, size_t workspace_bytes,
                       void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (batch < 0 || seqlen < 0 || dim <= 0 || !(scale >= 0.f) || !(scale < INFINITY))
        return SSD_ERR_SHAPE;
    if (!gated_sizes(batch, seqlen, dim)) return SSD_ERR_UNSUPPORTED;
    if (batch == 0) return SSD_OK;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (!al(init_state, 4) || !al(final_state, 4) || !al(states, 4)) return SSD_ERR_ALIGN;
    if (seqlen == 0) {
        if (final_state && final_state != init_state) {
            const int64_t n = batch * dim;
            hipLaunchKernelGGL(k_gated_copy, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                               final_state, init_state, n);
            if (hipGetLastError() != hipSuccess) return SSD_ERR_HIP;
        }
        return SSD_OK;
    }
    if (!x || !gates || !lam || !y) return SSD_ERR_NULL;
    if (!io_aligned(io_dtype, x, gates, y) || !al(lam, 4) || !al(seq_idx, 4)) return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < gated_ws(batch, seqlen, dim, 2)) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    GArgs g{};
    g.x = x, g.gates = gates, g.lam = lam, g.scale = scale, g.init = init_state, g.seq = seq_idx;
    g.y = y, g.fin = final_state, g.states = states;
    g.b = batch, g.l = seqlen, g.d = dim, g.tiles = (seqlen + kGT - 1) / kGT;
    g.A = static_cast<float *>(workspace);
    g.S = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                    gated_ws(batch, seqlen, dim, 1));
    const int v = lanes(io_dtype, dim, final_state, states, x, gates, y);
    const hipError_t e = io_dtype == SSD_BF16
                             ? (v == 4 ? fwd<bf16, 4>(g, s) : v == 2 ? fwd<bf16, 2>(g, s)
                                                                     : fwd<bf16, 1>(g, s))
                             : (v == 4 ? fwd<float, 4>(g, s) : v == 2 ? fwd<float, 2>(g, s)
                                                                      : fwd<float, 1>(g, s));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

int32_t ssd_gated_scan_bwd(const void *x, const void *gates, const float *lam, float scale,
                           const float *init_state, const int32_t *seq_idx, const float *states,
                           const void *dy, const float *d_final, void *dx, void *dgates,
                           float *dlam, float *d_init, int64_t batch, int64_t seqlen, int64_t dim,
                           int32_t io_dtype, void *workspace, size_t workspace_bytes,
                           void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (batch <= 0 || seqlen <= 0 || dim <= 0 || !(scale >= 0.f) || !(scale < INFINITY))
        return SSD_ERR_SHAPE;
    if (!gated_sizes(batch, seqlen, dim)) return SSD_ERR_UNSUPPORTED;
    if (!x || !gates || !lam || !dy || !dx || !dgates || !dlam) return SSD_ERR_NULL;
    if (!io_aligned(io_dtype, x, gates, dy, dx, dgates) || !al(lam, 4) || !al(init_state, 4) ||
        !al(seq_idx, 4) || !al(states, 4) || !al(d_final, 4) || !al(dlam, 4) || !al(d_init, 4))
        return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < gated_ws(batch, seqlen, dim, 4)) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    GArgs g{};
    g.x = x, g.gates = gates, g.lam = lam, g.scale = scale, g.init = init_state, g.seq = seq_idx;
    g.kept = states, g.dy = dy, g.dfin = d_final, g.y = dx, g.dgates = dgates, g.fin = d_init;
    g.b = batch, g.l = seqlen, g.d = dim, g.tiles = (seqlen + kGT - 1) / kGT;
    char *ws = static_cast<char *>(workspace);
    const size_t one = gated_ws(batch, seqlen, dim, 1);
    g.A = reinterpret_cast<float *>(ws);
    g.S = reinterpret_cast<float *>(ws + one);
    g.R = reinterpret_cast<float *>(ws + 2 * one);
    g.part = reinterpret_cast<float *>(ws + 3 * one);
    const int v = lanes(io_dtype, dim, d_init, nullptr, x, gates, dy, dx, dgates);
    const hipError_t e =
        io_dtype == SSD_BF16
            ? (v == 4 ? bwd<bf16, 4>(g, dlam, s) : v == 2 ? bwd<bf16, 2>(g, dlam, s)
                                                          : bwd<bf16, 1>(g, dlam, s))
            : (v == 4 ? bwd<float, 4>(g, dlam, s) : v == 2 ? bwd<float, 2>(g, dlam, s)
                                                           : bwd<float, 1>(g, dlam, s));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

int32_t ssd_gated_step(float *state, const void *x, const void *gates, const float *lam,
                       float scale, void *y, int64_t batch, int64_t dim, int32_t io_dtype,
                       void *hip_stream) {
    if (io_dtype != SSD_F32 && io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (batch < 0 || dim <= 0 || !(scale >= 0.f) || !(scale < INFINITY)) return SSD_ERR_SHAPE;
    if (!gated_sizes(0, 0, dim) || batch > ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
    if (batch == 0) return SSD_OK;
    if (!state || !x || !gates || !lam || !y) return SSD_ERR_NULL;
    if (!al(state, 4) || !al(lam, 4) || !io_aligned(io_dtype, x, gates, y)) return SSD_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int v = lanes(io_dtype, dim, state, lam, x, gates, y);
    const int64_t n = batch * (dim / v), blocks = (n + 255) / 256;
    if (blocks > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
#define SSD_GSTEP(IO, VV)                                                                         \
    hipLaunchKernelGGL((k_gated_step<IO, VV>), dim3((unsigned)blocks), dim3(256), 0, s, state,    \
                       static_cast<const IO *>(x), static_cast<const IO *>(gates), lam, scale,    \
                       static_cast<IO *>(y), batch, dim)
    if (io_dtype == SSD_BF16) {
        if (v == 4) SSD_GSTEP(bf16, 4);
        else if (v == 2) SSD_GSTEP(bf16, 2);
        else SSD_GSTEP(bf16, 1);
    } else {
        if (v == 4) SSD_GSTEP(float, 4);
        else if (v == 2) SSD_GSTEP(float, 2);
        else SSD_GSTEP(float, 1);
    }
#undef SSD_GSTEP
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // extern "C"
