// The gated linear recurrence, per channel c of x [b, l, d]:
//
//   u_t = scale softplus(lam_c) sigmoid(r_t)     a_t = e^{-u_t}
//   h_t = a_t h_{t-1} + v_t,  v_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t,  y_t = h_t
//
// with r_t = gates[.., c] and i_t = gates[.., d + c] raw (before their
// sigmoids), its gradient, and one decode step of it.
//
// A tile is SEG * NW tokens of 64 * V channels: a lane owns V channels, each of
// the workgroup's NW waves a run of SEG consecutive tokens, so every load of a wave is one
// contiguous piece of a token's row.  A run is the map h -> A h + S of the
// state entering it (A = prod a_t, S its result from zero); runs compose in
// order: waves through LDS inside a tile, tiles through the workspace.
#include <hip/hip_runtime.h>

#include <math.h>

#include "../../include/ssd.h"
#include "ssd_device.hpp"

// Products and sums are fused only where the code says so: every lane width
// then gives the same bits.
#pragma clang fp contract(off)

namespace ssd {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

template <typename IO, int V> struct alignas(sizeof(IO) * V) VecIO { IO e[V]; };
template <int V> struct alignas(4 * V) VecF { float e[V]; };

__device__ __forceinline__ float sigmoid_f(float z) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(-z * kLog2e));
}

// softplus(v) = max(v, 0) + log1p(y), y = e^-|v|: the exponential with the
// rounding of its argument put back, and log1p(y) = 2 atanh(z), z = y / (2 + y)
// <= 1/3, from seven terms (the eighth is below 2^-26 of the sum).  Beyond 200 y
// is zero in fp32 whatever v, also for an infinite one (a NaN stays one).
__device__ __forceinline__ float softplus_f(float v) {
    const float w = v > 200.f || v < -200.f ? -200.f : -fabsf(v), p = w * kLog2e;
    // log2(e) = kLog2e + 1.9e-8
    const float lo = fmaf(w, kLog2e, -p) + w * 1.925963033e-8f;
    const float y = exp2_fast(p) * fmaf(lo, kLn2, 1.f);
    const float z = y * __builtin_amdgcn_rcpf(2.f + y), q = z * z;
    float s = fmaf(q, 1.f / 13, 1.f / 11);
    s = fmaf(q, s, 1.f / 9);
    s = fmaf(q, s, 1.f / 7);
    s = fmaf(q, s, 1.f / 5);
    s = fmaf(q, s, 1.f / 3);
    return fmaxf(v, 0.f) + 2.f * fmaf(z * q, s, z);
}

// scale softplus(lam) in binary orders.  A rate without bound (an infinite lam,
// or an overflow) is the largest finite value: its decay is zero all the same,
// and its products with a zero are zero and not NaN (a NaN stays one).
__device__ __forceinline__ float rate_of(float lam, float scale) {
    constexpr float kMost = 0x1.fffffep127f;
    const float s = softplus_f(lam), m = scale * (s > kMost ? kMost : s) * kLog2e;
    return m > kMost ? kMost : m;
}

// a = e^-u and 1 - a^2 = -expm1(-2u) for u = u2 ln 2 >= 0.  Where the
// subtraction would cancel (2u < 1/8) the difference is u2 times the cubic of
// least largest relative error (1.6e-8 there, before rounding); above, the
// subtraction loses at most three bits of fp32.
__device__ __forceinline__ void decay(float u2, float &a, float &om) {
    a = exp2_fast(-u2);
    const float s = u2 * fmaf(u2, fmaf(u2, fmaf(u2, -0.1463926534f, 0.4436125999f),
                                       -0.9608984357f), 1.386294340f);
    const float m = fmaf(-a, a, 1.f);
    om = u2 < 0.09016844f ? s : m;
}

// How the tiles of one column (64 V channels of one sequence) hand states
// along in one pass.  A tile publishes its own map as soon as its rows are
// read; a tile then needs the maps of the earlier tiles of its group and the
// state after the group before, which the last tile of that group publishes.
// So a state crosses a group per hand-over, and each sum has one order whatever
// runs first.  Tiles are numbered as their workgroups start (a ticket per
// column): every tile waits only for lower tickets of its own column, which are
// running and wait for lower ones in turn, so every wait ends.
//
// A channel's map is one 64-bit word (its A with the sign bit set, which A
// never has, and its S), a state one with a mark beside it: a word that is not
// zero is whole, so nothing has to be ordered against anything and a reader
// waits on the data itself (with a flag behind the data the writer waited for
// its stores and the reader made two trips: 65536 tokens of 64 channels 58
// against 49 us, the gradient of 3 x 1001 x 771 40 against 33).  Words are written and read at agent scope, as the XCDs' L2 caches are not
// coherent inside a kernel, and cleared before every call.
constexpr int kMostGroup = 32;    // tiles of a group: 8 to 32, see group_of
constexpr int kTicketWords = 32;  // a 128-byte line per column's ticket

struct Chain {
    uint32_t *ticket;  // [cols][kTicketWords]
    uint64_t *map;     // [cols][tiles][64 V]
    uint64_t *after;   // [cols][groups][64 V] the state after the group
    float *rate;       // [d] scale softplus(lam) in binary orders (NULL without a chain)
};

struct GArgs {
    const void *x, *gates;
    const float *lam;
    float scale;
    const float *init;
    const int32_t *seq;
    const float *kept;    // backward: states after every SSD_GATED_CHUNK tokens
    const void *dy;       // backward
    const float *dfin;    // backward
    void *y;              // forward output (NULL: states only), or dx
    void *dgates;
    float *fin;           // final state, or d_init
    float *states;        // forward output: states after every SSD_GATED_CHUNK tokens
    float *part;          // backward: per tile sums behind dlam [b, tiles, d]
    Chain ch;
    int64_t b, l, d, tiles, ncol;
    int group;  // tiles of a group
};

template <int V> struct Words { uint64_t e[V]; };

__device__ __forceinline__ void put_word(uint64_t *p, uint32_t lo, float hi) {
    __hip_atomic_store(p, ((uint64_t)__builtin_bit_cast(uint32_t, hi) << 32) | lo, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float word_value(uint64_t w) {
    return __builtin_bit_cast(float, (uint32_t)(w >> 32));
}
__device__ __forceinline__ float word_decay(uint64_t w) {
    return __builtin_bit_cast(float, (uint32_t)w & 0x7fffffffu);
}
// Waits until the V words at every lane's p are there.  The bound (many seconds)
// only turns a broken promise of the scheduler into NaN results instead of a hang.
template <int V> __device__ __forceinline__ Words<V> wait_words(const uint64_t *p) {
    Words<V> w;
    for (uint32_t n = 0; n < (1u << 25); ++n) {
        bool there = true;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w.e[e] = __hip_atomic_load(p + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            there = there && w.e[e] != 0;
        }
        if (__all(there)) return w;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) w.e[e] = 0x7fc000007fc00000ull;
    return w;
}

// What one tile's loads need: this lane's channels and its rows.
template <typename IO, int V, int SEG> struct Tile {
    uint32_t c;      // first channel of this lane (clamped to a valid one)
    bool live;       // the lane's channels exist
    int64_t row0;    // the sequence's first row in [b * l]
    int64_t t0;      // the wave's first token
    __device__ Tile(const GArgs &g, int64_t col, int64_t tile, int tokens) {
        const int lane = threadIdx.x & 63;
        c = ((uint32_t)col % (uint32_t)g.ncol * 64 + lane) * V;
        live = c < g.d;
        if (!live) c = 0;
        row0 = (int64_t)((uint32_t)col / (uint32_t)g.ncol) * g.l;
        t0 = tile * tokens + wave_id() * SEG;
    }
};

// V elements at element `row` + `lane` of p.  With the row wave-uniform and the
// lane's channel apart, the access is a scalar address plus a 32-bit offset
// (the forward pass at 65536 x 2560: 291 us, 296 with whole addresses).
template <typename IO, int V>
__device__ __forceinline__ VecIO<IO, V> ldv(const void *p, int64_t row, uint32_t lane = 0) {
    const char *q = reinterpret_cast<const char *>(static_cast<const IO *>(p) + row);
    return *reinterpret_cast<const VecIO<IO, V> *>(q + lane * (uint32_t)sizeof(IO));
}
template <typename IO, int V>
__device__ __forceinline__ void stv(void *p, int64_t row, uint32_t lane, const VecIO<IO, V> &v) {
    char *q = reinterpret_cast<char *>(static_cast<IO *>(p) + row);
    *reinterpret_cast<VecIO<IO, V> *>(q + lane * (uint32_t)sizeof(IO)) = v;
}

// The wave's rows of x, r and i (rows past the end read the last row).
template <typename IO, int V, int SEG> struct Rows {
    VecIO<IO, V> x[SEG], r[SEG], i[SEG];
    __device__ void load(const GArgs &g, const Tile<IO, V, SEG> &w) {
#pragma unroll
        for (int k = 0; k < SEG; ++k) {
            int64_t t = w.t0 + k;
            if (t >= g.l) t = g.l - 1;
            const int64_t row = (w.row0 + t) * g.d;
            x[k] = ldv<IO, V>(g.x, row, w.c);
            r[k] = ldv<IO, V>(g.gates, 2 * row, w.c);
            i[k] = ldv<IO, V>(g.gates, 2 * row + g.d, w.c);
        }
    }
};

// PACKED calls hold several documents a sequence.  A run that holds a document's
// first token keeps nothing of the state entering it, whatever that is: another
// document's infinity or NaN times zero would not be zero.  Its A is infinite,
// which no product of decays is, and says so (a zero would not do: decays that
// underflow are to pass a NaN of their document).  The selects of these two and of
// the tokens cost 1 to 8% of a call (65536 tokens of 64 channels 52 against 48
// us), so calls without documents are kernels without them.
constexpr float kCut = __builtin_inff();
// The state behind a run that h enters.
template <bool PACKED> __device__ __forceinline__ float through(float A, float S, float h) {
    return PACKED && A == kCut ? S : fmaf(A, h, S);
}
// A of two runs.
template <bool PACKED> __device__ __forceinline__ float join(float A, float B) {
    return PACKED && (A == kCut || B == kCut) ? kCut : A * B;
}

// Which of the wave's tokens (a bit each) start a document inside the sequence.
// Lane k reads token k's document and the one before it ahead of the rows, so
// that nothing waits for them later.
template <bool PACKED, int SEG> struct Starts {
    int here, before;
    template <typename W> __device__ __forceinline__ void load(const GArgs &g, const W &w) {
        here = before = 0;
        if (!PACKED) return;
        const int lane = threadIdx.x & 63;
        const int64_t t = w.t0 + lane;
        if (lane >= SEG || t <= 0 || t >= g.l) return;
        here = g.seq[w.row0 + t];
        before = g.seq[w.row0 + t - 1];
    }
    __device__ __forceinline__ uint32_t bits() const {
        return PACKED ? (uint32_t)__ballot(here != before) : 0;
    }
};

// The identity past the end.
template <typename IO, int V, int SEG>
__device__ __forceinline__ void mask(const GArgs &g, const Tile<IO, V, SEG> &w,
                                     float (&a)[SEG][V], float (&v)[SEG][V]) {
    if (w.t0 + SEG <= g.l) return;
#pragma unroll
    for (int k = 0; k < SEG; ++k) {
        const bool in = w.t0 + k < g.l;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            a[k][e] = in ? a[k][e] : 1.f;
            v[k][e] = in ? v[k][e] : 0.f;
        }
    }
}

// Decay and added value of the wave's tokens.
template <typename IO, int V, int SEG>
__device__ __forceinline__ void terms(const GArgs &g, const Tile<IO, V, SEG> &w,
                                      const Rows<IO, V, SEG> &rw, const float (&m2)[V],
                                      float (&a)[SEG][V], float (&v)[SEG][V]) {
#pragma unroll
    for (int k = 0; k < SEG; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float om;
            decay(m2[e] * sigmoid_f(to_f32(rw.r[k].e[e])), a[k][e], om);
            v[k][e] = __builtin_amdgcn_sqrtf(om) * sigmoid_f(to_f32(rw.i[k].e[e])) *
                      to_f32(rw.x[k].e[e]);
        }
        // a row's temporaries are dead before the next row's begin: without
        // this the scheduler interleaves the rows and spills
        __builtin_amdgcn_sched_barrier(0);
    }
    mask(g, w, a, v);
}

// The map of the wave's tokens.
template <int V, int SEG>
__device__ __forceinline__ void run_map(const float (&a)[SEG][V], const float (&v)[SEG][V],
                                        uint32_t cut, VecF<V> &A, VecF<V> &S) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float p = 1.f, s = 0.f;
        if (cut) {
            p = kCut;
#pragma unroll
            for (int k = 0; k < SEG; ++k) s = fmaf(a[k][e], cut >> k & 1 ? 0.f : s, v[k][e]);
        } else {
#pragma unroll
            for (int k = 0; k < SEG; ++k) {
                p *= a[k][e];
                s = fmaf(a[k][e], s, v[k][e]);
            }
        }
        A.e[e] = p;
        S.e[e] = s;
    }
}

template <typename IO, int V, int SEG>
__device__ __forceinline__ void rates(const GArgs &g, const Tile<IO, V, SEG> &w, float (&m2)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e)
        m2[e] = g.ch.rate ? g.ch.rate[w.c + e] : rate_of(g.lam[w.c + e], g.scale);
}

// This workgroup's tile of its column, in the order of the chain.
__device__ __forceinline__ int64_t take_ticket(const GArgs &g, int64_t col, uint32_t *slot) {
    if (threadIdx.x == 0)
        *slot = __hip_atomic_fetch_add(g.ch.ticket + col * kTicketWords, 1u, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*slot);
}

template <int V, int NW> struct Lds {
    VecF<V> A[NW][64], S[NW][64];             // the waves' maps
    VecF<V> pA[kMostGroup][64], pS[kMostGroup][64];     // the maps of the group's earlier tiles
    VecF<V> before[64];                         // the state after the group before
    uint32_t slot;
};

// Composes the tile's waves (in chain order: BACK takes them from the last),
// publishes, gathers what is before the tile and leaves the state entering it
// in h.  `first`: the state entering the chain, at the lane's channels (NULL:
// zero); the tiles that take it have read it before they publish anything, so
// the chain's end may overwrite it.  Every wave of the workgroup
// calls it; the waves' maps are in lds.A, lds.S already.
template <int V, int NW, bool BACK, bool PACKED>
__device__ __forceinline__ void enter_tile(const GArgs &g, Lds<V, NW> &lds, int64_t col, int64_t j,
                                           const float *first, float (&h)[V]) {
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int grp = (int)j / g.group, in = (int)j % g.group;
    const int64_t groups = (g.tiles + g.group - 1) / g.group;
    const bool last = in == g.group - 1 && j + 1 < g.tiles;
    constexpr int W = 64 * V;
    if (wv == NW - 1 && grp == 0) {
        VecF<V> p;
#pragma unroll
        for (int e = 0; e < V; ++e) p.e[e] = first ? first[e] : 0.f;
        lds.before[lane] = p;
    }
    __syncthreads();
    VecF<V> tA, tS;
    if (wv == 0 && j + 1 < g.tiles) {
#pragma unroll
        for (int e = 0; e < V; ++e) tA.e[e] = 1.f, tS.e[e] = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const VecF<V> A = lds.A[BACK ? NW - 1 - k : k][lane];
            const VecF<V> S = lds.S[BACK ? NW - 1 - k : k][lane];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                tA.e[e] = join<PACKED>(tA.e[e], A.e[e]);
                tS.e[e] = through<PACKED>(A.e[e], S.e[e], tS.e[e]);
            }
        }
        if (!last) {
            uint64_t *m = g.ch.map + (col * g.tiles + j) * W + lane * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                put_word(m + e, __builtin_bit_cast(uint32_t, tA.e[e]) | 0x80000000u, tS.e[e]);
        }
    }
    // the earlier tiles of the group, a wave each; the group before by the last wave
    for (int k = wv; k < in; k += NW) {
        const int64_t t = (int64_t)grp * g.group + k;
        const Words<V> m = wait_words<V>(g.ch.map + (col * g.tiles + t) * W + lane * V);
        VecF<V> A, S;
#pragma unroll
        for (int e = 0; e < V; ++e) A.e[e] = word_decay(m.e[e]), S.e[e] = word_value(m.e[e]);
        lds.pA[k][lane] = A;
        lds.pS[k][lane] = S;
    }
    if (wv == NW - 1 && grp > 0) {
        const Words<V> m = wait_words<V>(g.ch.after + (col * groups + grp - 1) * W + lane * V);
        VecF<V> p;
#pragma unroll
        for (int e = 0; e < V; ++e) p.e[e] = word_value(m.e[e]);
        lds.before[lane] = p;
    }
    __syncthreads();
    const VecF<V> p = lds.before[lane];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = p.e[e];
    for (int k = 0; k < in; ++k) {
        const VecF<V> A = lds.pA[k][lane], S = lds.pS[k][lane];
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = through<PACKED>(A.e[e], S.e[e], h[e]);
    }
    if (wv == 0 && last) {
        uint64_t *m = g.ch.after + (col * groups + grp) * W + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) put_word(m + e, 1, through<PACKED>(tA.e[e], tS.e[e], h[e]));
    }
    // the waves before this one
#pragma unroll
    for (int k = 0; k < NW - 1; ++k) {
        const int w = BACK ? NW - 1 - k : k;
        if (BACK ? w > wv : w < wv) {
            const VecF<V> A = lds.A[w][lane], S = lds.S[w][lane];
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] = through<PACKED>(A.e[e], S.e[e], h[e]);
        }
    }
}

// Clears the words of one or two chains (counts of 16 bytes), and works out the
// channels' rates once (a softplus is as much work as a token's decay).
__global__ __launch_bounds__(256) void k_gated_setup(u32x4 *p, int64_t n, u32x4 *p2, int64_t n2,
                                                     const float *lam, float scale, float *rate,
                                                     int64_t d) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    const u32x4 zero = {0, 0, 0, 0};
    for (int64_t i = k; i < n; i += all) p[i] = zero;
    for (int64_t i = k; i < n2; i += all) p2[i] = zero;
    for (int64_t i = k; i < d; i += all) rate[i] = rate_of(lam[i], scale);
}

// ------------------------------------------------------------- forward ----
// One pass: 8 bytes an element (bf16).  65536 x 2560: 291 us, 4.6 TB/s; without
// the chain (a probe) the same loads, arithmetic and stores take 237, so what is
// left is the hand-over.  Reading everything twice (maps, chain, states) took
// 857.  A wave takes 16 tokens of 128 channels in bf16: with 8 of 256 the tiles'
// maps are twice the traffic (350 us).
template <typename IO, int V, int SEG, int NW, bool PACKED>
__global__ __launch_bounds__(NW * 64, 4) void k_gated_fwd(GArgs g) {
    constexpr int T = SEG * NW;
    static_assert(T % SSD_GATED_CHUNK == 0 && SSD_GATED_CHUNK % SEG == 0, "where states are kept");
    __shared__ Lds<V, NW> lds;
    const int lane = threadIdx.x & 63, wv = wave_id();
    const uint32_t cols = (uint32_t)(g.b * g.ncol);
    const int64_t col = blockIdx.x % cols;
    const int64_t tile = g.tiles > 1 ? take_ticket(g, col, &lds.slot) : 0;
    const Tile<IO, V, SEG> w(g, col, tile, T);
    const int64_t bi = (uint32_t)col / (uint32_t)g.ncol;
    Starts<PACKED, SEG> st;
    st.load(g, w);
    float m2[V];
    rates(g, w, m2);
    Rows<IO, V, SEG> rw;
    rw.load(g, w);
    const float *first = g.init ? g.init + bi * g.d + w.c : nullptr;
    float a[SEG][V], v[SEG][V];
    const uint32_t cut = st.bits();
    terms(g, w, rw, m2, a, v);
    VecF<V> A, S;
    run_map(a, v, cut, A, S);
    lds.A[wv][lane] = A;
    lds.S[wv][lane] = S;
    float h[V];
    enter_tile<V, NW, false, PACKED>(g, lds, col, tile, first, h);
    if (!w.live || w.t0 >= g.l) return;
#pragma unroll
    for (int k = 0; k < SEG; ++k) {
        const int64_t t = w.t0 + k;
        VecIO<IO, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (cut >> k & 1) h[e] = 0.f;
            h[e] = fmaf(a[k][e], h[e], v[k][e]);
            o.e[e] = (IO)h[e];
        }
        if (g.y && t < g.l) stv<IO, V>(g.y, (w.row0 + t) * g.d, w.c, o);
    }
    const int64_t end = w.t0 + SEG < g.l ? w.t0 + SEG : g.l;
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
//
// The states come from the forward pass's (or one more run of it), the adjoint
// is chained as the states are there.  14 bytes an element (bf16): 4 x 4096 x
// 2560 in 144 us, 4.1 TB/s.  Two workgroups a compute unit leave 128 registers
// a thread: four values an element are kept and 1 - a^2 is computed twice, which
// is one exponential more and no spilled registers (fp32: 2; five values kept:
// 12 and 169 us).  4 tokens a wave (more composing) take 187 us, 128-token tiles
// of 16 waves 159, 16 tokens a wave with one workgroup a unit 172.
template <typename IO, int V, int SEG, int NW, bool PACKED>
__global__ __launch_bounds__(NW * 64, 4) void k_gated_bwd(GArgs g) {
    constexpr int T = SEG * NW;
    static_assert(T % SSD_GATED_CHUNK == 0 && SSD_GATED_CHUNK % SEG == 0, "where states are kept");
    __shared__ Lds<V, NW> lds;
    __shared__ VecF<V> sS[NW][64];  // the waves' maps of the states; A is the adjoint's too
    const int lane = threadIdx.x & 63, wv = wave_id();
    const uint32_t cols = (uint32_t)(g.b * g.ncol);
    const int64_t col = blockIdx.x % cols, bi = (uint32_t)col / (uint32_t)g.ncol;
    // the chain runs from the last tile to the first
    const int64_t turn = g.tiles > 1 ? take_ticket(g, col, &lds.slot) : 0;
    const int64_t tile = g.tiles - 1 - turn;
    const Tile<IO, V, SEG> w(g, col, tile, T);
    Starts<PACKED, SEG> st;
    st.load(g, w);
    float m2[V];
    rates(g, w, m2);
    Rows<IO, V, SEG> rw;
    rw.load(g, w);
    VecIO<IO, V> dy[SEG];
#pragma unroll
    for (int k = 0; k < SEG; ++k) {
        const int64_t t = w.t0 + k < g.l ? w.t0 + k : g.l - 1;
        dy[k] = ldv<IO, V>(g.dy, (w.row0 + t) * g.d, w.c);
    }
    float h[V], q[V];
    const float *first = g.dfin ? g.dfin + bi * g.d + w.c : nullptr;
    const int64_t ns = (g.l + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int64_t ch = w.c + e;
        h[e] = tile > 0 ? g.kept[(bi * ns + tile * T / SSD_GATED_CHUNK - 1) * g.d + ch]
                        : (g.init ? g.init[bi * g.d + ch] : 0.f);
    }
    // kept for the second half: the decay and both gates
    float a[SEG][V], v[SEG][V], sr[SEG][V], si[SEG][V];
#pragma unroll
    for (int k = 0; k < SEG; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            sr[k][e] = sigmoid_f(to_f32(rw.r[k].e[e]));
            si[k][e] = sigmoid_f(to_f32(rw.i[k].e[e]));
            float om;
            decay(m2[e] * sr[k][e], a[k][e], om);
            v[k][e] = __builtin_amdgcn_sqrtf(om) * si[k][e] * to_f32(rw.x[k].e[e]);
        }
        __builtin_amdgcn_sched_barrier(0);  // as in terms()
    }
    const uint32_t cut = st.bits();
    mask(g, w, a, v);
    VecF<V> A, S, R;
    run_map(a, v, cut, A, S);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float r = 0.f;
#pragma unroll
        for (int k = SEG - 1; k >= 0; --k) {
            if (w.t0 + k < g.l) r = a[k][e] * (to_f32(dy[k].e[e]) + r);
            if (cut >> k & 1) r = 0.f;
        }
        R.e[e] = r;
    }
    lds.A[wv][lane] = A;
    lds.S[wv][lane] = R;
    sS[wv][lane] = S;
    enter_tile<V, NW, true, PACKED>(g, lds, col, turn, first, q);
#pragma unroll
    for (int j = 0; j < NW; ++j)
        if (j < wv) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                h[e] = through<PACKED>(lds.A[j][lane].e[e], sS[j][lane].e[e], h[e]);
        }
    __syncthreads();
    // the states before every token, in place of the added values
#pragma unroll
    for (int k = 0; k < SEG; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (cut >> k & 1) h[e] = 0.f;
            const float hn = fmaf(a[k][e], h[e], v[k][e]);
            v[k][e] = h[e];
            h[e] = hn;
        }
    VecF<V> acc;
#pragma unroll
    for (int e = 0; e < V; ++e) acc.e[e] = 0.f;
#pragma unroll
    for (int k = SEG - 1; k >= 0; --k) {
        const int64_t t = w.t0 + k;
        if (t >= g.l) continue;
        VecIO<IO, V> ox, orr, oi;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float x = to_f32(rw.x[k].e[e]), gt = to_f32(dy[k].e[e]) + q[e];
            // 1 - a^2 once more from the gate: the compiler, which would keep
            // the first one and spill, is not to see that they are the same
            asm volatile("" : "+v"(sr[k][e]));
            const float u2 = m2[e] * sr[k][e];
            // at: a[k][e].  The gradient takes a^2 from it: 1 - om, om being
            // rounded near one, is off by 2e-3 of itself at u = 5.5 and has
            // nothing left from u = 9
            float at, om;
            decay(u2, at, om);
            // 1 / beta; a shut gate (om = 0) has a finite stand-in for it, which
            // u = 0 then cancels
            const float rb = __builtin_amdgcn_rsqf(fmaxf(om, 0x1p-126f));
            const float gx = gt * si[k][e], gb = gx * __builtin_amdgcn_sqrtf(om), gbx = gb * x;
            q[e] = cut >> k & 1 ? 0.f : a[k][e] * gt;
            const float p = kLn2 * u2 * fmaf(at * at * rb, gx * x, -q[e] * v[k][e]);
            ox.e[e] = (IO)gb;
            oi.e[e] = (IO)fmaf(-gbx, si[k][e], gbx);
            orr.e[e] = (IO)fmaf(-p, sr[k][e], p);
            acc.e[e] += p;
        }
        __builtin_amdgcn_sched_barrier(0);
        if (w.live) {
            const int64_t row = (w.row0 + t) * g.d;
            stv<IO, V>(g.y, row, w.c, ox);
            stv<IO, V>(g.dgates, 2 * row, w.c, orr);
            stv<IO, V>(g.dgates, 2 * row + g.d, w.c, oi);
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
        for (int j = 0; j < NW; ++j) s.e[e] += sS[j][lane].e[e];
    }
    *reinterpret_cast<VecF<V> *>(g.part + (bi * g.tiles + tile) * g.d + w.c) = s;
    if (g.fin && tile == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) s.e[e] = q[e];
        *reinterpret_cast<VecF<V> *>(g.fin + bi * g.d + w.c) = s;
    }
}

// dlam: the tiles' sums, added in a fixed order in fp64.  One workgroup: 32
// channels by 32 runs of tiles, sixteen loads in flight a thread.
__global__ __launch_bounds__(1024) void k_gated_lam(const float *part, const float *lam,
                                                    float *dlam, int64_t rows, int64_t d) {
    __shared__ double s[32][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t ch = (int64_t)blockIdx.x * 32 + c;
    double t = 0;
    if (ch < d) {
        int64_t j = k;
        for (; j + 32 * 15 < rows; j += 512) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = part[(j + 32 * i) * d + ch];
#pragma unroll
            for (int i = 0; i < 16; ++i) t += v[i];
        }
        for (; j + 96 < rows; j += 128) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = part[(j + 32 * i) * d + ch];
#pragma unroll
            for (int i = 0; i < 4; ++i) t += v[i];
        }
        for (; j < rows; j += 32) t += part[j * d + ch];
    }
    s[k][c] = t;
    __syncthreads();
    if (k != 0 || ch >= d) return;
#pragma unroll
    for (int j = 1; j < 32; ++j) t += s[j][c];
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
    const uint32_t q = (uint32_t)d / V, k = blockIdx.x * 256 + threadIdx.x;  // fewer than 2^32
    if (k >= b * q) return;
    const int64_t bi = k / q, c = (int64_t)(k % q) * V, at = bi * d + c;
    VecF<V> h = *reinterpret_cast<const VecF<V> *>(state + at);
    const VecF<V> lm = *reinterpret_cast<const VecF<V> *>(lam + c);
    const VecIO<IO, V> xv = ldv<IO, V>(x, at), r = ldv<IO, V>(gates, at + bi * d),
                       i = ldv<IO, V>(gates, at + (bi + 1) * d);
    VecIO<IO, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float a, om;
        decay(rate_of(lm.e[e], scale) * sigmoid_f(to_f32(r.e[e])), a, om);
        h.e[e] = fmaf(a, h.e[e], __builtin_amdgcn_sqrtf(om) * sigmoid_f(to_f32(i.e[e])) *
                                     to_f32(xv.e[e]));
        o.e[e] = (IO)h.e[e];
    }
    *reinterpret_cast<VecF<V> *>(state + at) = h;
    stv<IO, V>(y, at, 0, o);
}

// batch > 0, seqlen == 0: the final state is the initial one, or zeros
__global__ __launch_bounds__(256) void k_gated_copy(float *dst, const float *src, int64_t n) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
        dst[k] = src ? src[k] : 0.f;
}

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int kLeastTile = 64;  // tokens of the shortest tile

// Workspace: a chain's tickets, maps and states after groups for any lane width
// (the gradient may need a second one, to run the forward pass), the rates, and
// for the gradient the states it starts from and the sums behind dlam.
struct GatedWs {
    size_t chain, chain2, rate, kept, part, total;
    GatedWs(int64_t b, int64_t l, int64_t d, bool bwd) {
        auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
        const int64_t tiles = (l + kLeastTile - 1) / kLeastTile, groups = (tiles + 7) / 8;
        const int64_t cols = b * ((d + 63) / 64), wide = b * ((d + 255) / 256 * 256);
        const bool one = tiles == 1;
        const size_t words = one ? 0 : up(cols * kTicketWords * 4 + wide * (tiles + groups) * 8);
        size_t o = 0;
        chain = o, o += words;
        chain2 = o, o += bwd ? words : 0;
        rate = o, o += one ? 0 : up((size_t)d * 4);
        kept = o, o += bwd && !one ? up((size_t)b * ((l + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK) * d * 4) : 0;
        part = o, o += bwd ? up((size_t)b * tiles * d * 4) : 0;
        total = o > 256 ? o : 256;
    }
};

// Channels a lane moves at once: `most` (4 or 2) or 2 where the width and every tensor allow
// vector accesses of as many elements, else 1.
template <typename... P> int lanes(int io, int64_t d, int most, const float *f0,
                                   const float *f1, P... p) {
    for (int v = most; v > 1; v /= 2) {
        const uintptr_t a = v * (io == SSD_BF16 ? 2 : 4), f = 4 * v;
        if (d % v == 0 && al(f0, f) && al(f1, f) && (al(p, a) && ...))
            return v;
    }
    return 1;
}
template <typename... P> bool io_aligned(int io, P... p) {
    return (al(p, io == SSD_BF16 ? 2 : 4) && ...);
}

// Sizes whose workgroups (of 512 threads) and threads are counted in 32 bits.
bool gated_sizes(int64_t b, int64_t l, int64_t d) {
    return b <= 65535 && d <= ((int64_t)1 << 24) && l <= ((int64_t)1 << 28) &&
           b * ((d + 63) / 64) * ((l + kLeastTile - 1) / kLeastTile) < ((int64_t)1 << 23);
}

// Tokens per wave and waves per workgroup of the two passes.
template <typename IO> struct FwdShape { static constexpr int SEG = sizeof(IO) == 2 ? 16 : 8, NW = 8; };
struct BwdShape { static constexpr int SEG = 8, NW = 8; };

// Tiles of a group.  A column's states cross a group per hand-over (2-3 us),
// and each tile reads the maps of half a group: where few columns or few tiles
// leave the chain of hand-overs to wait for, long groups are better (65536
// tokens of 64 channels: 58 us with 32, 125 with 8), with many the maps are
// traffic (2560 channels: 318 against 295).
int group_of(int64_t cols, int64_t tiles) {
    return cols <= 4 || cols * tiles <= 1024 ? 32 : cols <= 12 ? 16 : 8;
}

// The layout of a chain at lane width v and `tokens` a tile, in `words`; returns
// the 16-byte pieces to clear.
int64_t set_chain(GArgs &g, char *words, float *rate, int v, int tokens) {
    g.ncol = (g.d + 64 * v - 1) / (64 * v);
    g.tiles = (g.l + tokens - 1) / tokens;
    const int64_t cols = g.b * g.ncol;
    g.group = group_of(cols, g.tiles);  // a call of one tile divides by it too
    if (g.tiles == 1) return 0;
    const int64_t groups = (g.tiles + g.group - 1) / g.group;
    g.ch.ticket = reinterpret_cast<uint32_t *>(words);
    g.ch.map = reinterpret_cast<uint64_t *>(words + cols * kTicketWords * 4);
    g.ch.after = g.ch.map + cols * g.tiles * 64 * v;
    g.ch.rate = rate;
    return cols * (kTicketWords * 4 + (g.tiles + groups) * 64 * v * 8) / 16;
}

void setup(const GArgs &g, char *words, int64_t n, char *words2, int64_t n2, float *rate,
           hipStream_t s) {
    if (n + n2 == 0) return;
    int64_t blocks = ((n > g.d ? n : g.d) + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(k_gated_setup, dim3((unsigned)blocks), dim3(256), 0, s,
                       reinterpret_cast<u32x4 *>(words), n, reinterpret_cast<u32x4 *>(words2), n2,
                       g.lam, g.scale, rate, g.d);
}

template <typename IO, int V> void run_fwd(const GArgs &g, hipStream_t s) {
    typedef FwdShape<IO> F;
    const dim3 grid((unsigned)(g.b * g.ncol * g.tiles)), block(F::NW * 64);
    if (g.seq)
        hipLaunchKernelGGL((k_gated_fwd<IO, V, F::SEG, F::NW, true>), grid, block, 0, s, g);
    else
        hipLaunchKernelGGL((k_gated_fwd<IO, V, F::SEG, F::NW, false>), grid, block, 0, s, g);
}

template <typename IO, int V>
hipError_t fwd(GArgs g, const GatedWs &W, char *ws, hipStream_t s) {
    typedef FwdShape<IO> F;
    float *rate = reinterpret_cast<float *>(ws + W.rate);
    const int64_t n = set_chain(g, ws + W.chain, rate, V, F::SEG * F::NW);
    setup(g, ws + W.chain, n, nullptr, 0, rate, s);
    run_fwd<IO, V>(g, s);
    return hipGetLastError();
}

template <typename IO, int V>
hipError_t bwd(GArgs g, const GatedWs &W, char *ws, float *dlam, hipStream_t s) {
    typedef BwdShape B;
    typedef FwdShape<IO> F;
    float *rate = reinterpret_cast<float *>(ws + W.rate);
    const int64_t n = set_chain(g, ws + W.chain, rate, V, B::SEG * B::NW);
    if (!g.kept && g.tiles > 1) {  // the states that the tiles start from
        GArgs f = g;
        f.ch = Chain{};
        f.y = nullptr, f.fin = nullptr, f.states = reinterpret_cast<float *>(ws + W.kept);
        const int64_t n2 = set_chain(f, ws + W.chain2, rate, V, F::SEG * F::NW);
        setup(g, ws + W.chain, n, ws + W.chain2, n2, rate, s);
        run_fwd<IO, V>(f, s);
        g.kept = f.states;
    } else {
        setup(g, ws + W.chain, n, nullptr, 0, rate, s);
    }
    const dim3 grid((unsigned)(g.b * g.ncol * g.tiles)), block(B::NW * 64);
    if (g.seq)
        hipLaunchKernelGGL((k_gated_bwd<IO, V, B::SEG, B::NW, true>), grid, block, 0, s, g);
    else
        hipLaunchKernelGGL((k_gated_bwd<IO, V, B::SEG, B::NW, false>), grid, block, 0, s, g);
    hipLaunchKernelGGL(k_gated_lam, dim3((unsigned)((g.d + 31) / 32)), dim3(1024), 0, s, g.part,
                       g.lam, dlam, g.b * g.tiles, g.d);
    return hipGetLastError();
}

}  // namespace

}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_gated_scan_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
    if (batch <= 0 || seqlen <= 0 || dim <= 0 || !gated_sizes(batch, seqlen, dim)) return 0;
    return GatedWs(batch, seqlen, dim, false).total;
}

size_t ssd_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
    if (batch <= 0 || seqlen <= 0 || dim <= 0 || !gated_sizes(batch, seqlen, dim)) return 0;
    return GatedWs(batch, seqlen, dim, true).total;
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
            const unsigned blocks = (unsigned)(n < 65536 * 256 ? (n + 255) / 256 : 65536);
            hipLaunchKernelGGL(k_gated_copy, dim3(blocks), dim3(256), 0, s, final_state, init_state,
                               n);
            if (hipGetLastError() != hipSuccess) return SSD_ERR_HIP;
        }
        return SSD_OK;
    }
    if (!x || !gates || !lam || !y) return SSD_ERR_NULL;
    if (!io_aligned(io_dtype, x, gates, y) || !al(lam, 4) || !al(seq_idx, 4)) return SSD_ERR_ALIGN;
    const GatedWs W(batch, seqlen, dim, false);
    if (!workspace || workspace_bytes < W.total) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    GArgs g{};
    g.x = x, g.gates = gates, g.lam = lam, g.scale = scale, g.init = init_state, g.seq = seq_idx;
    g.y = y, g.fin = final_state, g.states = states;
    g.b = batch, g.l = seqlen, g.d = dim;
    char *ws = static_cast<char *>(workspace);
    const int v = lanes(io_dtype, dim, 2, final_state, states, x, gates, y);
    const hipError_t e = io_dtype == SSD_BF16
                             ? (v == 2 ? fwd<bf16, 2>(g, W, ws, s) : fwd<bf16, 1>(g, W, ws, s))
                             : (v == 2 ? fwd<float, 2>(g, W, ws, s) : fwd<float, 1>(g, W, ws, s));
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
    const GatedWs W(batch, seqlen, dim, true);
    if (!workspace || workspace_bytes < W.total) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    GArgs g{};
    g.x = x, g.gates = gates, g.lam = lam, g.scale = scale, g.init = init_state, g.seq = seq_idx;
    g.kept = states, g.dy = dy, g.dfin = d_final, g.y = dx, g.dgates = dgates, g.fin = d_init;
    g.b = batch, g.l = seqlen, g.d = dim;
    char *ws = static_cast<char *>(workspace);
    g.part = reinterpret_cast<float *>(ws + W.part);
    const int v = lanes(io_dtype, dim, 2, d_init, nullptr, x, gates, dy, dx, dgates);
    const hipError_t e =
        io_dtype == SSD_BF16
            ? (v == 2 ? bwd<bf16, 2>(g, W, ws, dlam, s) : bwd<bf16, 1>(g, W, ws, dlam, s))
            : (v == 2 ? bwd<float, 2>(g, W, ws, dlam, s) : bwd<float, 1>(g, W, ws, dlam, s));
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
    const int v = lanes(io_dtype, dim, 4, state, lam, x, gates, y);
    const int64_t n = batch * (dim / v), blocks = (n + 255) / 256;
    if (n > ((int64_t)1 << 32) - 256) return SSD_ERR_UNSUPPORTED;
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
