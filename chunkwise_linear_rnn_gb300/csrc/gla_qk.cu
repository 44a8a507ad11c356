// gla_qk.cu — norms of the query and key rows with the rotation by position, in
// one pass from the token-major layout to the head-first one:
//     y = R_p(w * x * r),   r = 1 / sqrt(sum_i x_i^2 / n + eps),
// and its backward: with z = R_p^T dy, g = w * z and unit = x r,
//     dw = sum over rows of z * unit,   dx = r (g - unit * <g, unit> / n).
//
// One warp takes one row (a token's head); a lane takes every 32nd value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gla.h"
#include "gla_internal.h"

namespace gla {
namespace {

constexpr int kPartials = 608;   // thread blocks of the backward, at most (4 for each of 152 SMs)

struct QkArgs {
    const void *x[2];        // q, k
    const float *w[2];
    const void *dy[2];       // backward: gradients of the outputs
    void *y[2];              // forward: outputs; backward: grad_q, grad_k
    const long long *pos;
    const double *inv_freq;
    float *partial;          // backward with weights: [blocks][2][d]
    gla_qk_layout lay;
    int B, T, H[2], d, rot, interleaved;
    float inv_n, eps;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// A frequency as 2^64ths of a turn per position, without its whole turns: the
// angle of any whole position is then a product modulo 2^64, with no error but
// the frequency's own rounding times the position.
__device__ __forceinline__ unsigned long long turn_of(double inv_freq) {
    const double two64 = 18446744073709551616.0;
    const double inv_2pi = 0.15915494309189535, inv_2pi_low = -9.839338337591243e-18;   // 1 / (2 pi), in two parts
    const double f = inv_freq * inv_2pi;
    const double low = fma(inv_freq, inv_2pi, -f) + inv_freq * inv_2pi_low;
    return static_cast<unsigned long long>(__double2ll_rn((f - rint(f)) * two64)) +
           static_cast<unsigned long long>(__double2ll_rn(low * two64));
}

__device__ __forceinline__ void angle(unsigned long long turn, long long pos, float *c, float *s) {
    const long long a = static_cast<long long>(turn * static_cast<unsigned long long>(pos));
    // the top 32 bits, a signed fraction of half a turn in [-1, 1)
    sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f, s, c);
}

// Element i's partner in its pair, the pair's number, and +1 for a second member.
__device__ __forceinline__ int partner(const QkArgs &p, int i, int *pair, bool *second) {
    if (p.interleaved) {
        *pair = i >> 1;
        *second = i & 1;
        return i ^ 1;
    }
    *second = i >= p.rot / 2;
    *pair = *second ? i - p.rot / 2 : i;
    return *second ? i - p.rot / 2 : i + p.rot / 2;
}

struct Row {
    int which, h, b, t;
};

__device__ __forceinline__ Row row_of(const QkArgs &p, long long r) {
    const int heads = p.H[0] + p.H[1];
    Row o;
    const int h = static_cast<int>(r % heads);
    const long long token = r / heads;
    o.which = h >= p.H[0];
    o.h = o.which ? h - p.H[0] : h;
    o.b = static_cast<int>(token / p.T);
    o.t = static_cast<int>(token % p.T);
    return o;
}

template <typename E>
__device__ __forceinline__ const E *row_in(const QkArgs &p, const Row &o) {
    const E *x = static_cast<const E *>(p.x[o.which]);
    return o.which ? x + o.b * p.lay.k_sb + o.t * p.lay.k_st + o.h * p.lay.k_sh
                   : x + o.b * p.lay.q_sb + o.t * p.lay.q_st + o.h * p.lay.q_sh;
}

__device__ __forceinline__ size_t row_head_first(const QkArgs &p, const Row &o) {
    return ((static_cast<size_t>(o.b) * p.H[o.which] + o.h) * p.T + o.t) * p.d;
}

__device__ __forceinline__ long long position_of(const QkArgs &p, const Row &o) {
    return p.pos ? p.pos[o.b * p.lay.pos_sb + o.t] : o.t;
}

template <typename E>
__global__ void __launch_bounds__(256) qk_fwd_kernel(const __grid_constant__ QkArgs p,
                                                     long long rows) {
    const int lane = threadIdx.x & 31;
    for (long long r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < rows; r += gridDim.x * 8LL) {
        const Row o = row_of(p, r);
        const E *x = row_in<E>(p, o);
        const float *w = p.w[o.which];
        E *y = static_cast<E *>(p.y[o.which]) + row_head_first(p, o);
        const long long pos = position_of(p, o);
        float sum = 0.f;
        for (int i = lane; i < p.d; i += 32) sum = fmaf(to_f32(x[i]), to_f32(x[i]), sum);
        const float rn = 1.f / sqrtf(fmaf(warp_sum(sum), p.inv_n, p.eps));
        for (int i = lane; i < p.d; i += 32) {
            float v = to_f32(x[i]) * rn * (w ? w[i] : 1.f);
            if (i < p.rot) {
                int pair;
                bool second;
                const int j = partner(p, i, &pair, &second);
                const float u = to_f32(x[j]) * rn * (w ? w[j] : 1.f);
                float c, s;
                angle(turn_of(p.inv_freq[pair]), pos, &c, &s);
                v = second ? fmaf(u, s, v * c) : fmaf(-u, s, v * c);
            }
            put(y + i, v);
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(256) qk_bwd_kernel(const __grid_constant__ QkArgs p,
                                                     long long rows) {
    __shared__ float s_dw[8][2][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float dw[2][8] = {};
    for (long long r = blockIdx.x * 8LL + warp; r < rows; r += gridDim.x * 8LL) {
        const Row o = row_of(p, r);
        const E *x = row_in<E>(p, o);
        const float *w = p.w[o.which];
        const E *dy = static_cast<const E *>(p.dy[o.which]) + row_head_first(p, o);
        E *dx = static_cast<E *>(p.y[o.which]) +
                ((static_cast<size_t>(o.b) * p.T + o.t) * p.H[o.which] + o.h) * p.d;
        const long long pos = position_of(p, o);
        float sum = 0.f, dot = 0.f, z[8], xv[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const int i = lane + 32 * m;
            z[m] = xv[m] = 0.f;
            if (i >= p.d) continue;
            xv[m] = to_f32(x[i]);
            z[m] = to_f32(dy[i]);
            if (i < p.rot) {
                int pair;
                bool second;
                const int j = partner(p, i, &pair, &second);
                const float u = to_f32(dy[j]);
                float c, s;
                angle(turn_of(p.inv_freq[pair]), pos, &c, &s);
                z[m] = second ? fmaf(-u, s, z[m] * c) : fmaf(u, s, z[m] * c);
            }
            sum = fmaf(xv[m], xv[m], sum);
            dot = fmaf(z[m] * (w ? w[i] : 1.f), xv[m], dot);
        }
        const float rn = 1.f / sqrtf(fmaf(warp_sum(sum), p.inv_n, p.eps));
        const float back = warp_sum(dot) * rn * p.inv_n;   // <g, unit> / n
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const int i = lane + 32 * m;
            if (i >= p.d) continue;
            const float unit = xv[m] * rn;
            if (o.which) dw[1][m] = fmaf(z[m], unit, dw[1][m]);
            else dw[0][m] = fmaf(z[m], unit, dw[0][m]);
            put(dx + i, rn * (z[m] * (w ? w[i] : 1.f) - unit * back));
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        s_dw[warp][0][lane + 32 * m] = dw[0][m];
        s_dw[warp][1][lane + 32 * m] = dw[1][m];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.d; i += 256) {
        float v = 0.f;
        for (int k = 0; k < 8; ++k) v += s_dw[k][i / p.d][i % p.d];
        p.partial[static_cast<size_t>(blockIdx.x) * 2 * p.d + i] = v;
    }
}

// The blocks' partial weight gradients, added in order in fp64.
__global__ void __launch_bounds__(64) qk_weight_grad_kernel(const float *partial, int blocks, int d,
                                                            float *gq, float *gk) {
    const int i = blockIdx.x * 64 + threadIdx.x;
    if (i >= 2 * d) return;
    double v = 0.0;
    for (int b = 0; b < blocks; ++b) v += partial[static_cast<size_t>(b) * 2 * d + i];
    float *g = i < d ? gq + i : gk + (i - d);
    if (i < d ? gq != nullptr : gk != nullptr) *g = static_cast<float>(v);
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check(const QkArgs &a, const gla_qk_options &op) {
    for (int i = 0; i < 2; ++i)
        if (!aligned(a.x[i], 16) || !aligned(a.w[i], 16) || !aligned(a.dy[i], 16) ||
            !aligned(a.y[i], 16))
            return GLA_ERR_ARG;
    if (!aligned(a.pos, 8) || !aligned(a.inv_freq, 8)) return GLA_ERR_ARG;
    if (a.B <= 0 || a.T <= 0 || a.H[0] <= 0 || a.H[1] <= 0 || a.d <= 0 || a.rot < 0)
        return GLA_ERR_ARG;
    if (static_cast<long long>(a.H[0]) + a.H[1] > 0x7fffffffLL) return GLA_ERR_ARG;
    if (op.dtype != GLA_BF16 && op.dtype != GLA_F32) return GLA_ERR_ARG;
    if (op.norm != GLA_NORM_RMS && op.norm != GLA_NORM_L2) return GLA_ERR_ARG;
    if (op.interleaved != 0 && op.interleaved != 1) return GLA_ERR_ARG;
    if (!(op.eps > 0.f && op.eps <= 1.f)) return GLA_ERR_ARG;
    for (long long s : {a.lay.q_sb, a.lay.q_st, a.lay.q_sh, a.lay.k_sb, a.lay.k_st, a.lay.k_sh})
        if (s < 0 || s % 8) return GLA_ERR_ARG;
    if (a.lay.pos_sb < 0) return GLA_ERR_ARG;
    if (a.d % 8 || a.d > 256 || a.rot % 8 || a.rot > a.d) return GLA_ERR_SHAPE;
    if (a.rot > 0 && !a.inv_freq) return GLA_ERR_ARG;
    return GLA_OK;
}

void bind(QkArgs *a, const void *q, const void *k, const float *wq, const float *wk,
          const long long *positions, const double *inv_freq, void *y_q, void *y_k, int B, int T,
          int Hq, int Hk, int d, int rot, const gla_qk_layout &lay, const gla_qk_options &op) {
    a->x[0] = q;
    a->x[1] = k;
    a->w[0] = wq;
    a->w[1] = wk;
    a->y[0] = y_q;
    a->y[1] = y_k;
    a->pos = positions;
    a->inv_freq = inv_freq;
    a->lay = lay;
    a->B = B;
    a->T = T;
    a->H[0] = Hq;
    a->H[1] = Hk;
    a->d = d;
    a->rot = rot;
    a->interleaved = op.interleaved;
    a->inv_n = op.norm == GLA_NORM_RMS ? 1.f / static_cast<float>(std::max(d, 1)) : 1.f;
    a->eps = op.eps;
}

}  // namespace
}  // namespace gla

extern "C" {

int gla_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk,
                         const long long *positions, const double *inv_freq, void *q_out,
                         void *k_out, int B, int T, int Hq, int Hk, int d, int rot,
                         const gla_qk_layout *layout, const gla_qk_options *options,
                         cudaStream_t stream) {
    using namespace gla;
    if (!q || !k || !q_out || !k_out || !layout || !options) return GLA_ERR_ARG;
    QkArgs a = {};
    bind(&a, q, k, wq, wk, positions, inv_freq, q_out, k_out, B, T, Hq, Hk, d, rot, *layout,
         *options);
    int st = check(a, *options);
    if (st != GLA_OK) return st;
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const long long rows = static_cast<long long>(B) * T * (Hq + Hk);
    const unsigned grid = static_cast<unsigned>(std::min<long long>((rows + 7) / 8, 16LL * sms));
    if (options->dtype == GLA_BF16) qk_fwd_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, rows);
    else qk_fwd_kernel<float><<<grid, 256, 0, stream>>>(a, rows);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

unsigned long gla_qk_norm_rope_bwd_scratch(int d) {
    return d > 0 ? static_cast<unsigned long>(gla::kPartials) * 2 * d * sizeof(float) : 0;
}

int gla_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk,
                         const long long *positions, const double *inv_freq, const void *d_q,
                         const void *d_k, void *grad_q, void *grad_k, float *grad_wq,
                         float *grad_wk, int B, int T, int Hq, int Hk, int d, int rot,
                         const gla_qk_layout *layout, const gla_qk_options *options,
                         void *scratch, unsigned long scratch_bytes, cudaStream_t stream) {
    using namespace gla;
    if (!q || !k || !d_q || !d_k || !grad_q || !grad_k || !layout || !options) return GLA_ERR_ARG;
    if ((grad_wq && !wq) || (grad_wk && !wk)) return GLA_ERR_ARG;
    QkArgs a = {};
    bind(&a, q, k, wq, wk, positions, inv_freq, grad_q, grad_k, B, T, Hq, Hk, d, rot, *layout,
         *options);
    a.dy[0] = d_q;
    a.dy[1] = d_k;
    int st = check(a, *options);
    if (st != GLA_OK) return st;
    const bool weights = grad_wq || grad_wk;
    if (weights) {
        if (!scratch || !aligned(scratch, 16)) return GLA_ERR_ARG;
        if (scratch_bytes < gla_qk_norm_rope_bwd_scratch(d)) return GLA_ERR_SCRATCH;
        if (!aligned(grad_wq, 4) || !aligned(grad_wk, 4)) return GLA_ERR_ARG;
        a.partial = static_cast<float *>(scratch);
    }
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const long long rows = static_cast<long long>(B) * T * (Hq + Hk);
    const unsigned grid = static_cast<unsigned>(std::min<long long>((rows + 7) / 8, kPartials));
    if (options->dtype == GLA_BF16) qk_bwd_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, rows);
    else qk_bwd_kernel<float><<<grid, 256, 0, stream>>>(a, rows);
    if (weights && cudaGetLastError() == cudaSuccess)
        qk_weight_grad_kernel<<<(2 * d + 63) / 64, 64, 0, stream>>>(a.partial, grid, d, grad_wq,
                                                                     grad_wk);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // extern "C"
