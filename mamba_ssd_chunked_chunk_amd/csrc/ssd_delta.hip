// The gated delta rule's entry points (argument checks, workspace) and its
// decode step.  The chunked kernels are in ssd_delta_scan.hip and
// ssd_delta_bwd.hip, the formulas in ssd_delta.hpp.
#include "ssd_delta.hpp"

#include <math.h>
#include <initializer_list>

#include "../../include/ssd.h"

namespace ssd {

namespace {

// One token.  A workgroup holds the state of one (batch, head) in registers, a
// thread four columns of R rows, so the state is read once and written once:
// both S^T k and S^T q are taken from the state in front, as
//   S'^T q = a S^T q + (k . q) u,   u = beta (v - a S^T k).
// Bound by memory: 256 x 80 states of 128 x 64 in 256 us, 5.2 TB/s (a large copy
// reaches 4.9).
template <typename IO, int N, int P> struct StepShape {
    static constexpr int LP = P / 4, RG = N < 256 / LP ? N : 256 / LP, R = N / RG;
    static constexpr int THREADS = LP * RG, WAVES = THREADS / 64;
};

struct DeltaStep {
    float *state;
    const void *q, *k, *v, *dt, *beta;
    const float *A, *bias;
    void *y;
    int64_t h, g;
    int softplus, norm;
    float scale, eps, lo, hi;
};

template <typename IO, int N, int P>
__global__ __launch_bounds__((StepShape<IO, N, P>::THREADS)) void k_delta_step(DeltaStep a) {
    typedef StepShape<IO, N, P> Sh;
    constexpr int LP = Sh::LP, RG = Sh::RG, R = Sh::R;
    __shared__ float kq[2][N];
    __shared__ f32x4 red[2][Sh::WAVES][LP];
    __shared__ float dot[Sh::WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cq = tid % LP, rg = tid / LP;
    const int64_t bh = blockIdx.x, bb = bh / a.h, hh = bh % a.h, gg = hh / (a.h / a.g);
    f32x4 *st = reinterpret_cast<f32x4 *>(a.state + bh * N * P) + cq;
    f32x4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = st[(rg + RG * i) * LP];
    if (wave < 2) {  // k, q: a wave each
        const IO *src = static_cast<const IO *>(wave ? a.q : a.k) + (bb * a.g + gg) * N;
        constexpr int E = N < 64 ? 1 : N / 64;
        float v[E], mx = 0.f, ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = lane + 64 * e < N ? to_f32(src[lane + 64 * e]) : 0.f;
            mx = fmaxf(mx, fabsf(v[e]));
        }
        float unit = 1.f;
        if (a.norm) {  // the norm of the row over its largest value stays in range
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
            const int ex = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) & 255;
            const float sc = __builtin_bit_cast(
                float, (uint32_t)(mx == 0.f ? 127 : 253 - ex < 1 ? 1 : 253 - ex) << 23);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= sc, ss = fmaf(v[e], v[e], ss);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) ss += __shfl_xor(ss, o);
            unit = UnitRow(ss, sc, 1.f / sc, a.eps).of_scaled;
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 64 * e < N) kq[wave][lane + 64 * e] = v[e] * unit;
    }
    const int64_t at = bb * a.h + hh;
    const float step = time_step(to_f32(static_cast<const IO *>(a.dt)[at]), a.bias ? a.bias[hh] : 0.f,
                                 a.softplus, a.lo, a.hi);
    const float keep = expf(fmaxf(a.A[hh] * step, -1e4f));
    const float beta = to_f32(static_cast<const IO *>(a.beta)[at]);
    const f32x4 v = ld4<IO>(static_cast<const IO *>(a.v) + bh * P + 4 * cq);
    __syncthreads();
    float kk[R];
    f32x4 sk = zero4(), sq = zero4();
    float kd = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        kk[i] = kq[0][rg + RG * i];
        const float q = kq[1][rg + RG * i];
        kd = fmaf(kk[i], q, kd);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk[e] = fmaf(S[i][e], kk[i], sk[e]);
            sq[e] = fmaf(S[i][e], q, sq[e]);
        }
    }
#pragma unroll
    for (int o = LP; o < 64; o <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sk[e] += __shfl_xor(sk[e], o), sq[e] += __shfl_xor(sq[e], o);
        kd += __shfl_xor(kd, o);
    }
    if (lane < LP) red[0][wave][lane] = sk, red[1][wave][lane] = sq;
    if (lane == 0) dot[wave] = kd;
    __syncthreads();
    sk = zero4(), sq = zero4(), kd = 0.f;
#pragma unroll
    for (int w = 0; w < Sh::WAVES; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sk[e] += red[0][w][cq][e], sq[e] += red[1][w][cq][e];
        kd += dot[w];
    }
    f32x4 u, y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        u[e] = beta * fmaf(-keep, sk[e], v[e]);
        y[e] = a.scale * fmaf(kd, u[e], keep * sq[e]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        f32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(kk[i], u[e], keep * S[i][e]);
        st[(rg + RG * i) * LP] = o;
    }
    if (rg == 0) st4<IO>(static_cast<IO *>(a.y) + bh * P + 4 * cq, y);
}

template <typename IO> hipError_t step_io(const DeltaStep &a, int64_t bh, int n, int p, hipStream_t s) {
#define SSD_CASE(NN, PP)                                                                      \
    if (n == NN && p == PP) {                                                                 \
        hipLaunchKernelGGL((k_delta_step<IO, NN, PP>), dim3((unsigned)bh),                    \
                           dim3(StepShape<IO, NN, PP>::THREADS), 0, s, a);                    \
        return hipGetLastError();                                                             \
    }
#define SSD_ROW(NN) SSD_CASE(NN, 16) SSD_CASE(NN, 32) SSD_CASE(NN, 64) SSD_CASE(NN, 128)
    SSD_ROW(32) SSD_ROW(64) SSD_ROW(128)
#undef SSD_ROW
#undef SSD_CASE
    return hipErrorInvalidValue;
}

__global__ void k_delta_copy(float *dst, const float *src, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        dst[i] = src ? src[i] : 0.f;
}

// ------------------------------------------------------------- workspace ---
struct DeltaWs {
    size_t total = 0, hbytes;
    size_t gimg, himg, rows2, nimg, zimg, simg, dsimg, yimg, scales, g0, x0, toks, eend, cells, part, states;
    size_t add(size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~(size_t)255;
        return at;
    }
    DeltaWs(int64_t b, int64_t l, int64_t h, int64_t n, int64_t p, int64_t g, int io, bool grad,
            bool keep) {
        const size_t el = io == SSD_BF16 ? 2 : 4, planes = el / 2;  // of k and q
        const size_t nc = (size_t)((l + kDC - 1) / kDC), ch = b * nc * h, cg = b * nc * g;
        const size_t tri = kPieces * 1024;
        gimg = add(cg * 2 * planes * kDC * n * 2);
        hbytes = 2 * tri + kRows * kDC * 4 + (grad ? 4 : 2) * tri;
        himg = add(ch * hbytes);
        rows2 = nimg = zimg = simg = dsimg = yimg = scales = g0 = x0 = toks = eend = cells = part = states = 0;
        if (!grad) return;
        rows2 = add(ch * kRowsGrad * kDC * 4);
        nimg = add(ch * kDC * p * 4);  // two fp16 terms or one fp32
        zimg = add(ch * kDC * p * 4);
        simg = add(ch * n * p * 4);
        dsimg = add(ch * n * p * 4);
        yimg = add(ch * kDC * p * el);
        scales = add(ch * (p / 16) * kScales * 4);
        g0 = add(ch * kDC * p * 4);
        x0 = add(ch * kDC * p * 4);
        toks = add(ch * (p / 16) * kSums * kDC * 4);
        eend = add(ch * (p / 16) * 4);
        cells = add(ch * 5 * kDC * 8);
        part = add(ch * 2 * 8);
        if (keep) states = add(ch * n * p * 4);
    }
    void set(DeltaArgs &a, char *ws, bool grad) const {
        a.gimg = ws + gimg, a.himg = ws + himg;
        a.hstride = hbytes;
        if (!grad) return;
        a.rows2 = reinterpret_cast<float *>(ws + rows2);
        a.nimg = ws + nimg, a.zimg = ws + zimg, a.simg = ws + simg, a.dsimg = ws + dsimg;
        a.yimg = ws + yimg;
        a.scales = reinterpret_cast<float *>(ws + scales);
        a.g0 = reinterpret_cast<float *>(ws + g0);
        a.x0 = reinterpret_cast<float *>(ws + x0);
        a.toks = reinterpret_cast<float *>(ws + toks);
        a.eend = reinterpret_cast<float *>(ws + eend);
        a.cells = reinterpret_cast<double *>(ws + cells);
        a.part = reinterpret_cast<double *>(ws + part);
    }
};

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool all_al(uintptr_t a, std::initializer_list<const void *> p) {
    for (const void *q : p)
        if (!al(q, a)) return false;
    return true;
}

bool delta_dims(int64_t p, int64_t n) {
    return (p == 16 || p == 32 || p == 64 || p == 128) && (n == 32 || n == 64 || n == 128);
}
// Sizes whose launches, 32-bit offsets inside 64 rows and counts stay in range.
bool delta_sizes(int64_t b, int64_t l, int64_t h) {
    return b <= 65535 && h <= 16384 && l <= ((int64_t)1 << 28) &&
           b * h * ((l + kDC - 1) / kDC) < ((int64_t)1 << 23);
}

int32_t delta_check(int64_t b, int64_t l, int64_t h, int64_t p, int64_t n, int64_t g, int io, float eps,
                    int norm) {
    if (io != SSD_F32 && io != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (b < 0 || l < 0 || h <= 0 || g <= 0 || p <= 0 || n <= 0 || h % g) return SSD_ERR_SHAPE;
    if (norm && !(eps >= 0.f && eps < INFINITY)) return SSD_ERR_SHAPE;
    if (!delta_dims(p, n)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

}  // namespace

}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_delta_scan_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t value_dim,
                                      int64_t key_dim, int64_t groups, int32_t io_dtype) {
    if (delta_check(batch, seqlen, heads, value_dim, key_dim, groups, io_dtype, 0.f, 0) != SSD_OK ||
        batch == 0 || seqlen == 0 || !delta_sizes(batch, seqlen, heads))
        return 0;
    return DeltaWs(batch, seqlen, heads, key_dim, value_dim, groups, io_dtype, false, false).total;
}

int32_t ssd_delta_scan(const void *q, const void *k, const void *v, const void *dt, const float *A,
                       const float *dt_bias, int32_t dt_softplus, float dt_min, float dt_max,
                       const void *beta, float scale, int32_t normalize, float norm_eps,
                       const float *init_state, const int32_t *seq_idx, void *y, float *final_state,
                       float *states, int64_t batch, int64_t seqlen, int64_t heads,
                       int64_t value_dim, int64_t key_dim, int64_t groups, int32_t io_dtype,
                       void *workspace, size_t workspace_bytes, void *hip_stream) {
    const int32_t bad = delta_check(batch, seqlen, heads, value_dim, key_dim, groups, io_dtype,
                                    norm_eps, normalize);
    if (bad != SSD_OK) return bad;
    if (!delta_sizes(batch, seqlen, heads)) return SSD_ERR_UNSUPPORTED;
    if (batch == 0) return SSD_OK;
    if (!all_al(16, {init_state, final_state, states})) return SSD_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (seqlen == 0) {
        if (final_state && final_state != init_state) {
            const int64_t n = batch * heads * key_dim * value_dim, blocks = (n + 255) / 256;
            hipLaunchKernelGGL(k_delta_copy, dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                               dim3(256), 0, s, final_state, init_state, n);
            if (hipGetLastError() != hipSuccess) return SSD_ERR_HIP;
        }
        return SSD_OK;
    }
    if (!q || !k || !v || !dt || !A || !beta || !y) return SSD_ERR_NULL;
    if (!all_al(16, {q, k, v, y}) || !all_al(4, {A, dt_bias, seq_idx}) ||
        !all_al(io_dtype == SSD_BF16 ? 2 : 4, {dt, beta}))
        return SSD_ERR_ALIGN;
    const DeltaWs W(batch, seqlen, heads, key_dim, value_dim, groups, io_dtype, false, false);
    if (!workspace || workspace_bytes < W.total) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    DeltaArgs a{};
    a.q = q, a.k = k, a.v = v, a.dt = dt, a.beta = beta, a.A = A, a.bias = dt_bias;
    a.init = init_state, a.seq = seq_idx, a.y = y, a.fin = final_state, a.states = states;
    a.b = batch, a.l = seqlen, a.h = heads, a.g = groups, a.nc = (seqlen + kDC - 1) / kDC;
    a.p = (int)value_dim, a.softplus = dt_softplus, a.norm = normalize;
    a.scale = scale, a.eps = norm_eps, a.lo = dt_min, a.hi = dt_max;
    W.set(a, static_cast<char *>(workspace), false);
    hipError_t e = delta_prep(a, io_dtype, (int)key_dim, false, s);
    if (e == hipSuccess) e = delta_forward(a, io_dtype, (int)key_dim, s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

size_t ssd_delta_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                          int64_t value_dim, int64_t key_dim, int64_t groups,
                                          int32_t io_dtype, int32_t with_states) {
    if (delta_check(batch, seqlen, heads, value_dim, key_dim, groups, io_dtype, 0.f, 0) != SSD_OK ||
        batch == 0 || seqlen == 0 || !delta_sizes(batch, seqlen, heads))
        return 0;
    return DeltaWs(batch, seqlen, heads, key_dim, value_dim, groups, io_dtype, true, !with_states)
        .total;
}

int32_t ssd_delta_scan_bwd(const void *q, const void *k, const void *v, const void *dt, const float *A,
                           const float *dt_bias, int32_t dt_softplus, float dt_min, float dt_max,
                           const void *beta, float scale, int32_t normalize, float norm_eps,
                           const float *init_state, const int32_t *seq_idx, const float *states,
                           const void *dy, const float *d_final, void *dq, void *dk, void *dv,
                           void *ddt, void *dbeta, float *dA, float *ddt_bias, float *d_init,
                           int64_t batch, int64_t seqlen, int64_t heads, int64_t value_dim,
                           int64_t key_dim, int64_t groups, int32_t io_dtype, void *workspace,
                           size_t workspace_bytes, void *hip_stream) {
    const int32_t bad = delta_check(batch, seqlen, heads, value_dim, key_dim, groups, io_dtype,
                                    norm_eps, normalize);
    if (bad != SSD_OK) return bad;
    if (batch == 0 || seqlen == 0) return SSD_ERR_SHAPE;
    if (!delta_sizes(batch, seqlen, heads)) return SSD_ERR_UNSUPPORTED;
    if (!q || !k || !v || !dt || !A || !beta || !dy || !dq || !dk || !dv || !ddt || !dbeta || !dA)
        return SSD_ERR_NULL;
    if (!all_al(16, {q, k, v, dy, dq, dk, dv, init_state, states, d_final, d_init}) ||
        !all_al(4, {A, dt_bias, seq_idx, dA, ddt_bias}) ||
        !all_al(io_dtype == SSD_BF16 ? 2 : 4, {dt, beta, ddt, dbeta}))
        return SSD_ERR_ALIGN;
    const DeltaWs W(batch, seqlen, heads, key_dim, value_dim, groups, io_dtype, true, !states);
    if (!workspace || workspace_bytes < W.total) return SSD_ERR_WORKSPACE;
    if (!al(workspace, 256)) return SSD_ERR_ALIGN;
    DeltaArgs a{};
    a.q = q, a.k = k, a.v = v, a.dt = dt, a.beta = beta, a.A = A, a.bias = dt_bias;
    a.init = init_state, a.seq = seq_idx, a.kept = states, a.dy = dy, a.dfin = d_final;
    a.dq = dq, a.dk = dk, a.dv = dv, a.ddt = ddt, a.dbeta = dbeta;
    a.dA = dA, a.dbias = ddt_bias, a.dinit = d_init;
    a.b = batch, a.l = seqlen, a.h = heads, a.g = groups, a.nc = (seqlen + kDC - 1) / kDC;
    a.p = (int)value_dim, a.softplus = dt_softplus, a.norm = normalize;
    a.scale = scale, a.eps = norm_eps, a.lo = dt_min, a.hi = dt_max;
    char *ws = static_cast<char *>(workspace);
    W.set(a, ws, true);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int n = (int)key_dim;
    if (!states) a.states = reinterpret_cast<float *>(ws + W.states);
    hipError_t e = delta_prep(a, io_dtype, n, true, s);
    if (!states) {
        a.y = a.nimg;  // not needed, nor right with these images: to where N comes later
        if (e == hipSuccess) e = delta_forward(a, io_dtype, n, s);
        a.kept = a.states;
    }
    if (e == hipSuccess) e = delta_backward(a, io_dtype, n, s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

int32_t ssd_delta_step(float *state, const void *q, const void *k, const void *v, const void *dt,
                       const float *A, const float *dt_bias, int32_t dt_softplus, float dt_min,
                       float dt_max, const void *beta, float scale, int32_t normalize, float norm_eps,
                       void *y, int64_t batch, int64_t heads, int64_t value_dim, int64_t key_dim,
                       int64_t groups, int32_t io_dtype, void *hip_stream) {
    const int32_t bad =
        delta_check(batch, 1, heads, value_dim, key_dim, groups, io_dtype, norm_eps, normalize);
    if (bad != SSD_OK) return bad;
    if (heads > 16384 || batch > ((int64_t)1 << 23) / heads) return SSD_ERR_UNSUPPORTED;
    if (batch == 0) return SSD_OK;
    if (!state || !q || !k || !v || !dt || !A || !beta || !y) return SSD_ERR_NULL;
    const uintptr_t el = io_dtype == SSD_BF16 ? 2 : 4;
    if (!al(state, 16) || !all_al(4 * el, {v, y}) || !all_al(4, {A, dt_bias}) ||
        !all_al(el, {q, k, dt, beta}))
        return SSD_ERR_ALIGN;
    DeltaStep a{};
    a.state = state, a.q = q, a.k = k, a.v = v, a.dt = dt, a.beta = beta, a.A = A, a.bias = dt_bias;
    a.y = y, a.h = heads, a.g = groups, a.softplus = dt_softplus, a.norm = normalize;
    a.scale = scale, a.eps = norm_eps, a.lo = dt_min, a.hi = dt_max;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int64_t bh = batch * heads;
    const hipError_t e = io_dtype == SSD_BF16 ? step_io<bf16>(a, bh, (int)key_dim, (int)value_dim, s)
                                              : step_io<float>(a, bh, (int)key_dim, (int)value_dim, s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // extern "C"
