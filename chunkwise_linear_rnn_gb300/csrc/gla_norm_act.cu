// gla_norm_act.cu — the norm of each head's channels with the activation that follows it
// (a group norm, channels last), and its gradients.  A row is one head of one token:
//     xhat = (x - mean) r,  n = xhat w + b,   y = n f(gate)  or  y = f(n),
// and backward, with dn = dy f(gate) (or dy f'(n)) and u = dn w:
//     dgate = dy n f'(gate),  dw = sum dn xhat,  db = sum dn,
//     dx = r (u - mean(u) - xhat mean(u xhat))     (mean(u) = 0 without the mean).
//
// A warp keeps its heads (a group of lanes and 8 or 16 values a lane for each) and walks
// tokens, so that weights and the sums for their gradients stay in registers, whether every
// head has its own or not.  Eight warps take eight neighbouring tokens: head-first rows of a
// block are then contiguous runs too.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "gla.h"
#include "gla_internal.h"
#include "gla_ptx.cuh"

namespace gla {
namespace {

constexpr int kWarps = 8;
constexpr long long kFwdBlocks = 4864;   // thread blocks of the forward, at most (32 an SM)
constexpr long long kBwdBlocks = 608;    // of the backward, where that keeps kSumRows (4 an SM)
constexpr int kSumRows = 1024;           // rows that a lane adds in 32 bits

struct NormArgs {
    const void *x, *gate, *dy;
    const float *w, *b;
    void *y, *dx, *dgate;
    float *partial;          // backward with weights: see reduce_kernel
    gla_norm_act_layout lay;
    unsigned tokens, T;      // T = tokens where one stride steps over batch and tokens
    int H, d, groups;        // groups of the heads that a warp takes together
    int layer, silu, per_channel;
    float inv_d, eps;
};

// Eight neighbouring values of a row, in 32 bits.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// s(z) = 1 / (1 + exp(-z)).  Rows that end in bf16 take the hardware's 2^x and reciprocal (each
// within a few roundings of 2^-23), fp32 rows CUDA's own.
__device__ __forceinline__ float sigmoid(float z, __nv_bfloat16) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2f(-1.4426950408889634f * z)));
    return r;
}
__device__ __forceinline__ float sigmoid(float z, float) { return 1.f / (1.f + expf(-z)); }

// A warp's place: its lanes' heads and channels.
template <int LANES, int NB>
struct Place {
    int h, group;
    bool there[NB];
    int c[NB];               // first channel of each of the lane's blocks of 8

    __device__ __forceinline__ Place(const NormArgs &p) {
        constexpr int ROWS = 32 / LANES;
        const int lane = threadIdx.x & 31, j = lane % LANES;
        group = blockIdx.x % p.groups;
        h = group * ROWS + lane / LANES;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            c[i] = 8 * (j + i * LANES);
            there[i] = h < p.H && c[i] < p.d;
        }
    }
};

template <int LANES, int NB>
__device__ __forceinline__ void load_weights(const NormArgs &p, const Place<LANES, NB> &at,
                                             float (&w)[NB][8], float (&b)[NB][8]) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = 1.f, b[i][e] = 0.f;
        if (!at.there[i]) continue;
        const int o = (p.per_channel ? at.h * p.d : 0) + at.c[i];
        if (p.w) load8(p.w + o, w[i]);
        if (p.b) load8(p.b + o, b[i]);
    }
}

// Where a token's row starts, in elements.
__device__ __forceinline__ long long row_of(const NormArgs &p, unsigned n, long long sb,
                                            long long st) {
    if (p.T == p.tokens) return n * st;
    const unsigned b = n / p.T;
    return b * sb + (n - b * p.T) * st;
}

// x becomes xhat; returns r.
template <int LANES, int NB>
__device__ __forceinline__ float normalise(const NormArgs &p, const Place<LANES, NB> &at,
                                           float (&x)[NB][8]) {
    if (p.layer) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[i][e];
        const float mean = group_sum<LANES>(s) * p.inv_d;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = at.there[i] ? x[i][e] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[i][e], x[i][e], s);
    const float r = rsqrtf(fmaf(group_sum<LANES>(s), p.inv_d, p.eps));
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= r;
    return r;
}

template <typename E, int LANES, int NB, bool GATE>
__global__ void __launch_bounds__(32 * kWarps) norm_fwd_kernel(const NormArgs p) {
    constexpr int U = NB == 1 ? 2 : 1;   // tokens whose loads are under way together
    const Place<LANES, NB> at(p);
    float w[NB][8], b[NB][8];
    load_weights<LANES, NB>(p, at, w, b);
    const unsigned step = gridDim.x / p.groups * kWarps * U;
    for (unsigned n0 = blockIdx.x / p.groups * kWarps * U + threadIdx.x / 32; n0 < p.tokens;
         n0 += step) {
        float x[U][NB][8], g[U][NB][8];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const unsigned n = n0 + k * kWarps;
            const bool real = n < p.tokens;
            const E *px = static_cast<const E *>(p.x) + row_of(p, n, p.lay.x_sb, p.lay.x_st) +
                          at.h * p.lay.x_sh;
            const E *pg = nullptr;
            if (GATE)
                pg = static_cast<const E *>(p.gate) + row_of(p, n, p.lay.g_sb, p.lay.g_st) +
                     at.h * p.lay.g_sh;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][i][e] = g[k][i][e] = 0.f;
                if (real && at.there[i]) {
                    load8(px + at.c[i], x[k][i]);
                    if (GATE) load8(pg + at.c[i], g[k][i]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const unsigned n = n0 + k * kWarps;
            normalise<LANES, NB>(p, at, x[k]);
            E *py = static_cast<E *>(p.y) +
                    (static_cast<long long>(n) * p.H + at.h) * p.d;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = fmaf(x[k][i][e], w[i][e], b[i][e]);
                    const float z = GATE ? g[k][i][e] : m;
                    const float s = sigmoid(z, E{});
                    const float f = p.silu ? z * s : s;
                    y[e] = GATE ? m * f : f;
                }
                if (n < p.tokens && at.there[i]) store8(py + at.c[i], y);
            }
        }
    }
}

// The sums of a block: over its warps in their order, and over the heads of a warp where they
// share a weight.  v: a lane's values; out: the block's row of the partial sums.
template <int LANES, int NB>
__device__ __forceinline__ void block_sums(const NormArgs &p, const Place<LANES, NB> &at,
                                           float (*buf)[32][NB][8], float (&v)[NB][8],
                                           float *out) {
    constexpr int ROWS = 32 / LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();   // the buffer's last use
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) buf[warp][lane][i][e] = v[i][e];
    __syncthreads();
    // one thread a value: per head [ROWS][d], or summed over the rows [d]
    const int values = p.per_channel ? ROWS * p.d : p.d;
    for (int c = threadIdx.x; c < values; c += 32 * kWarps) {
        const int r = c / p.d, ch = c - r * p.d, i = ch / 8 / LANES, j = ch / 8 % LANES;
        float s = 0.f;
        for (int row = r; row < (p.per_channel ? r + 1 : ROWS); ++row)
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += buf[k][row * LANES + j][i][ch % 8];
        out[c] = s;
    }
}

template <typename E, int LANES, int NB, bool GATE>
__global__ void __launch_bounds__(32 * kWarps) norm_bwd_kernel(const NormArgs p) {
    __shared__ float buf[kWarps][32][NB][8];
    const Place<LANES, NB> at(p);
    float w[NB][8], b[NB][8], dw[NB][8], db[NB][8];
    load_weights<LANES, NB>(p, at, w, b);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;
    const unsigned step = gridDim.x / p.groups * kWarps;
    for (unsigned n = blockIdx.x / p.groups * kWarps + threadIdx.x / 32; n < p.tokens; n += step) {
        float x[NB][8], g[NB][8], dy[NB][8];
        const E *px = static_cast<const E *>(p.x) + row_of(p, n, p.lay.x_sb, p.lay.x_st) +
                      at.h * p.lay.x_sh;
        const E *pg = nullptr;
        if (GATE)
            pg = static_cast<const E *>(p.gate) + row_of(p, n, p.lay.g_sb, p.lay.g_st) +
                 at.h * p.lay.g_sh;
        const long long flat = (static_cast<long long>(n) * p.H + at.h) * p.d;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = g[i][e] = dy[i][e] = 0.f;
            if (at.there[i]) {
                load8(px + at.c[i], x[i]);
                load8(static_cast<const E *>(p.dy) + flat + at.c[i], dy[i]);
                if (GATE) load8(pg + at.c[i], g[i]);
            }
        }
        const float r = normalise<LANES, NB>(p, at, x);
        float su = 0.f, sux = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float dg[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float m = fmaf(x[i][e], w[i][e], b[i][e]);
                const float z = GATE ? g[i][e] : m;
                const float s = sigmoid(z, E{});
                const float f = p.silu ? z * s : s;
                const float slope = p.silu ? s * fmaf(z, 1.f - s, 1.f) : s * (1.f - s);
                const float dn = dy[i][e] * (GATE ? f : slope);
                dg[e] = dy[i][e] * m * slope;
                dw[i][e] = fmaf(dn, x[i][e], dw[i][e]);
                db[i][e] += dn;
                const float u = dn * w[i][e];
                dy[i][e] = u;
                su += u;
                sux = fmaf(u, x[i][e], sux);
            }
            if (GATE && at.there[i]) store8(static_cast<E *>(p.dgate) + flat + at.c[i], dg);
        }
        const float m1 = group_sum<LANES>(sux) * p.inv_d;
        const float m0 = p.layer ? group_sum<LANES>(su) * p.inv_d : 0.f;
        E *pd = static_cast<E *>(p.dx) + row_of(p, n, p.lay.dx_sb, p.lay.dx_st) +
                at.h * p.lay.dx_sh;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r * (dy[i][e] - m0 - x[i][e] * m1);
            if (at.there[i]) store8(pd + at.c[i], v);
        }
    }
    if (p.partial) {
        constexpr int ROWS = 32 / LANES;
        const long long row = p.per_channel ? static_cast<long long>(ROWS) * p.d : p.d;
        float *out = p.partial + blockIdx.x * row;
        block_sums<LANES, NB>(p, at, buf, dw, out);
        block_sums<LANES, NB>(p, at, buf, db, out + gridDim.x * row);
    }
}

// The gradients of weight (blockIdx.y = 0) and bias from the blocks' sums, partial
// [2][blocks][values]: the values of blocks b, b + groups, ... belong to the same heads where
// each head has weights of its own (groups > 1 only there), else every block has the same ones.
// 32 channels of a block, one warp-wide row of 32 partial sums each; sums in fp64.
__global__ void __launch_bounds__(1024) reduce_kernel(const float *partial, unsigned blocks,
                                                      int groups, int values, int channels,
                                                      float *dw, float *db) {
    __shared__ double buf[32][33];
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    double s = 0.;
    if (c < channels) {
        const unsigned group = c / values;
        const float *from = partial + static_cast<size_t>(blockIdx.y) * blocks * values + c % values;
        for (unsigned k = group + ry * groups; k < blocks; k += 32 * groups)
            s += from[static_cast<size_t>(k) * values];
    }
    buf[ry][cx] = s;
    __syncthreads();
    if (ry == 0 && c < channels) {
        for (int k = 1; k < 32; ++k) s += buf[k][cx];
        out[c] = static_cast<float>(s);
    }
}

// ---------------------------------------------------------------- launches

// Heads that a warp takes together, by the lanes that a row of d values needs.
int rows_of(int d) { return d <= 64 ? 4 : d <= 128 ? 2 : 1; }

// Blocks for each group of heads: enough for the GPU, no more than there are tokens, and in the
// backward no fewer than keep a lane's sums to kSumRows rows.
long long token_blocks(long long tokens, int groups, int each, long long most, int sum_rows) {
    const long long want = std::min((tokens + kWarps * each - 1) / (kWarps * each),
                                    std::max(1LL, most / groups));
    return std::max(want, sum_rows ? (tokens + kWarps * sum_rows - 1) / (kWarps * sum_rows) : 1);
}

template <typename E, int LANES, int NB>
int launch_fwd(const NormArgs &a, cudaStream_t stream) {
    const long long tb = token_blocks(a.tokens, a.groups, NB == 1 ? 2 : 1, kFwdBlocks, 0);
    if (tb * a.groups > INT_MAX) return -1;
    const unsigned grid = static_cast<unsigned>(tb * a.groups);
    if (a.gate) norm_fwd_kernel<E, LANES, NB, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else norm_fwd_kernel<E, LANES, NB, false><<<grid, 32 * kWarps, 0, stream>>>(a);
    return static_cast<int>(cudaGetLastError());
}

template <typename E, int LANES, int NB>
int launch_bwd(const NormArgs &a, float *dw, float *db, cudaStream_t stream) {
    const long long tb = token_blocks(a.tokens, a.groups, 1, kBwdBlocks, kSumRows);
    if (tb * a.groups > INT_MAX) return -1;
    const unsigned grid = static_cast<unsigned>(tb * a.groups);
    if (a.gate) norm_bwd_kernel<E, LANES, NB, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else norm_bwd_kernel<E, LANES, NB, false><<<grid, 32 * kWarps, 0, stream>>>(a);
    if (a.partial) {
        const int channels = a.per_channel ? a.H * a.d : a.d;
        const int values = a.per_channel ? 32 / LANES * a.d : a.d;
        reduce_kernel<<<dim3((channels + 31) / 32, 2), 1024, 0, stream>>>(
            a.partial, grid, a.per_channel ? a.groups : 1, values, channels, dw, db);
    }
    return static_cast<int>(cudaGetLastError());
}

template <typename E>
int fwd(const NormArgs &a, cudaStream_t stream) {
    if (a.d <= 64) return launch_fwd<E, 8, 1>(a, stream);
    if (a.d <= 128) return launch_fwd<E, 16, 1>(a, stream);
    if (a.d <= 256) return launch_fwd<E, 32, 1>(a, stream);
    return launch_fwd<E, 32, 2>(a, stream);
}

template <typename E>
int bwd(const NormArgs &a, float *dw, float *db, cudaStream_t stream) {
    if (a.d <= 64) return launch_bwd<E, 8, 1>(a, dw, db, stream);
    if (a.d <= 128) return launch_bwd<E, 16, 1>(a, dw, db, stream);
    if (a.d <= 256) return launch_bwd<E, 32, 1>(a, dw, db, stream);
    return launch_bwd<E, 32, 2>(a, dw, db, stream);
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The arguments that both directions have, checked.
int bind(NormArgs *a, const void *x, const void *gate, const float *weight, const float *bias,
         int B, int T, int H, int d, const gla_norm_act_layout &lay,
         const gla_norm_act_options &op, bool backward) {
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(weight, 16) || !aligned(bias, 16))
        return GLA_ERR_ARG;
    if (B <= 0 || T <= 0 || H <= 0 || d <= 0) return GLA_ERR_ARG;
    if (op.dtype != GLA_BF16 && op.dtype != GLA_F32) return GLA_ERR_ARG;
    if (op.norm != GLA_NORM_RMS && op.norm != GLA_NORM_LAYER) return GLA_ERR_ARG;
    if (op.activation != GLA_ACT_SILU && op.activation != GLA_ACT_SIGMOID) return GLA_ERR_ARG;
    if (op.per_channel != 0 && op.per_channel != 1) return GLA_ERR_ARG;
    if (!(op.eps > 0.f && op.eps <= 1.f)) return GLA_ERR_ARG;
    for (long long s : {lay.x_sb, lay.x_st, lay.x_sh, lay.g_sb, lay.g_st, lay.g_sh})
        if (s < 0 || s % 8) return GLA_ERR_ARG;
    if (backward)
        for (long long s : {lay.dx_sb, lay.dx_st, lay.dx_sh})
            if (s < 0 || s % 8) return GLA_ERR_ARG;
    if (d % 8 || d > 512) return GLA_ERR_SHAPE;
    const long long tokens = static_cast<long long>(B) * T;
    // token numbers are counted on past the last in 32 bits, channels of all heads in 31
    if (tokens > INT_MAX || static_cast<long long>(H) * d > INT_MAX - 64) return GLA_ERR_ARG;
    *a = {};
    a->x = x;
    a->gate = gate;
    a->w = weight;
    a->b = bias;
    a->lay = lay;
    a->tokens = static_cast<unsigned>(tokens);
    a->T = static_cast<unsigned>(T);
    // one stride for all tokens: a single token a sequence, or sequences one behind the other
    gla_norm_act_layout &l = a->lay;
    if (T == 1) {
        l.x_st = l.x_sb, l.g_st = l.g_sb, l.dx_st = l.dx_sb;
        a->T = a->tokens;
    } else if (B == 1 || (l.x_sb == T * l.x_st && (!gate || l.g_sb == T * l.g_st) &&
                          (!backward || l.dx_sb == T * l.dx_st))) {
        a->T = a->tokens;
    }
    a->H = H;
    a->d = d;
    a->groups = (H + rows_of(d) - 1) / rows_of(d);
    a->layer = op.norm == GLA_NORM_LAYER;
    a->silu = op.activation == GLA_ACT_SILU;
    a->per_channel = op.per_channel;
    a->inv_d = 1.f / static_cast<float>(d);
    a->eps = op.eps;
    return GLA_OK;
}

}  // namespace
}  // namespace gla

extern "C" {

int gla_group_norm_act_fwd(const void *x, const void *gate, const float *weight,
                           const float *bias, void *y, int B, int T, int H, int d,
                           const gla_norm_act_layout *layout, const gla_norm_act_options *options,
                           cudaStream_t stream) {
    using namespace gla;
    if (!x || !y || !layout || !options || !aligned(y, 16)) return GLA_ERR_ARG;
    NormArgs a;
    int st = bind(&a, x, gate, weight, bias, B, T, H, d, *layout, *options, false);
    if (st != GLA_OK) return st;
    a.y = y;
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const int e = options->dtype == GLA_BF16 ? fwd<__nv_bfloat16>(a, stream) : fwd<float>(a, stream);
    return e == 0 ? GLA_OK : e < 0 ? GLA_ERR_ARG : GLA_ERR_LAUNCH;
}

unsigned long gla_group_norm_act_bwd_scratch(int B, int T, int H, int d) {
    using namespace gla;
    if (B <= 0 || T <= 0 || H <= 0 || d <= 0) return 0;
    const int rows = rows_of(d), groups = (H + rows - 1) / rows;
    const long long tb = token_blocks(static_cast<long long>(B) * T, groups, 1, kBwdBlocks, kSumRows);
    return 2ul * sizeof(float) * tb * groups * rows * d;
}

int gla_group_norm_act_bwd(const void *x, const void *gate, const float *weight,
                           const float *bias, const void *dy, void *grad_x, void *grad_gate,
                           float *grad_weight, float *grad_bias, int B, int T, int H, int d,
                           const gla_norm_act_layout *layout, const gla_norm_act_options *options,
                           void *scratch, unsigned long scratch_bytes, cudaStream_t stream) {
    using namespace gla;
    if (!x || !dy || !grad_x || !layout || !options) return GLA_ERR_ARG;
    if (!gate != !grad_gate || (grad_weight && !weight) || (grad_bias && !bias)) return GLA_ERR_ARG;
    if (!aligned(dy, 16) || !aligned(grad_x, 16) || !aligned(grad_gate, 16)) return GLA_ERR_ARG;
    NormArgs a;
    int st = bind(&a, x, gate, weight, bias, B, T, H, d, *layout, *options, true);
    if (st != GLA_OK) return st;
    a.dy = dy;
    a.dx = grad_x;
    a.dgate = grad_gate;
    if (grad_weight || grad_bias) {
        if (!scratch || !aligned(scratch, 16)) return GLA_ERR_ARG;
        if (scratch_bytes < gla_group_norm_act_bwd_scratch(B, T, H, d)) return GLA_ERR_SCRATCH;
        if (!aligned(grad_weight, 4) || !aligned(grad_bias, 4)) return GLA_ERR_ARG;
        a.partial = static_cast<float *>(scratch);
    }
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const int e = options->dtype == GLA_BF16
                      ? bwd<__nv_bfloat16>(a, grad_weight, grad_bias, stream)
                      : bwd<float>(a, grad_weight, grad_bias, stream);
    return e == 0 ? GLA_OK : e < 0 ? GLA_ERR_ARG : GLA_ERR_LAUNCH;
}

}  // extern "C"
