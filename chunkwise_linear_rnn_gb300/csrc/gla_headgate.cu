// gla_headgate.cu — prompts through the recurrence with one gate per token and head:
//     S_t = a_t S_{t-1} + k_t^T v_t,     o_t = scale q_t S_t,    a_t = exp(log_alpha_t),
// over a packed batch, token-major, with fewer key heads than value heads.
//
// Token by token: a thread holds one column of the state, a block 64 columns of one head of
// one sequence; the tokens' keys and queries come through shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "gla.h"
#include "gla_exp.cuh"
#include "gla_internal.h"
#include "gla_ptx.cuh"

namespace gla {

int headgate_check(const void *q, const void *k, const void *v, const float *log_alpha,
                   const float *h, const void *o, int Hk, int H, int dk, int dv,
                   const gla_headgate_layout &lay) {
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
          reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o) |
          reinterpret_cast<uintptr_t>(h)) & 15) ||
        (reinterpret_cast<uintptr_t>(log_alpha) & 3))
        return GLA_ERR_ARG;
    if (Hk <= 0 || H <= 0 || H > 65535 || H % Hk) return GLA_ERR_ARG;
    for (long long s : {lay.q_st, lay.q_sh, lay.k_st, lay.k_sh, lay.v_st, lay.v_sh})
        if (s < 0 || s % 8) return GLA_ERR_ARG;
    if (lay.a_st < 0 || lay.a_sh < 0) return GLA_ERR_ARG;
    if (dk <= 0 || dv <= 0 || dk % 8 || dv % 8 || dk > 128 || dv > 256) return GLA_ERR_SHAPE;
    return GLA_OK;
}

namespace {

constexpr int kBounds = 256;     // sequences of one launch

struct TokenArgs {
    const __nv_bfloat16 *q, *k, *v;
    const float *log_alpha, *h0;
    __nv_bfloat16 *o;
    float *hT;
    gla_headgate_layout lay;
    float scale;
    int H, share, dk, dv, first;
    int bounds[kBounds + 1];
};

constexpr int kMaxDk = 128, kCols = 64;

__global__ void __launch_bounds__(kCols) headgate_token_kernel(const __grid_constant__ TokenArgs p) {
    __shared__ float s_q[kMaxDk], s_k[kMaxDk];
    const int head = blockIdx.x, n = blockIdx.z, c = blockIdx.y * kCols + threadIdx.x;
    const int hk = head / p.share;
    const bool mine = c < p.dv;
    const long long state = ((static_cast<long long>(p.first + n) * p.H + head) * p.dk) * p.dv + c;
    float S[kMaxDk];
#pragma unroll
    for (int i = 0; i < kMaxDk; ++i)
        S[i] = p.h0 && mine && i < p.dk ? p.h0[state + static_cast<long long>(i) * p.dv] : 0.f;
    for (int i = threadIdx.x; i < kMaxDk; i += kCols) s_q[i] = s_k[i] = 0.f;
    for (int t = p.bounds[n]; t < p.bounds[n + 1]; ++t) {
        __syncthreads();
        for (int i = threadIdx.x; i < p.dk; i += kCols) {
            s_q[i] = __bfloat162float(p.q[t * p.lay.q_st + hk * p.lay.q_sh + i]);
            s_k[i] = __bfloat162float(p.k[t * p.lay.k_st + hk * p.lay.k_sh + i]);
        }
        const float a = exp_centred(p.log_alpha[t * p.lay.a_st + head * p.lay.a_sh]);
        const float v = mine ? __bfloat162float(p.v[t * p.lay.v_st + head * p.lay.v_sh + c]) : 0.f;
        __syncthreads();
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxDk; ++i) {
            S[i] = fmaf(a, S[i], s_k[i] * v);
            sum = fmaf(s_q[i], S[i], sum);
        }
        if (mine)
            p.o[(static_cast<long long>(t) * p.H + head) * p.dv + c] = __float2bfloat16_rn(p.scale * sum);
    }
    if (p.hT && mine)
#pragma unroll
        for (int i = 0; i < kMaxDk; ++i)
            if (i < p.dk) p.hT[state + static_cast<long long>(i) * p.dv] = S[i];
}

bool bounds_ok(const int *cu, int N, int T) {
    if (!cu || N <= 0 || T < 0 || cu[0] != 0 || cu[N] != T) return false;
    for (int n = 0; n < N; ++n)
        if (cu[n + 1] < cu[n]) return false;
    return true;
}

}  // namespace
}  // namespace gla

extern "C" {

unsigned long gla_headgate_fwd_varlen_scratch(const int *, int, int, int, int) { return 0; }

int gla_headgate_fwd_varlen(const void *q, const void *k, const void *v, const float *log_alpha,
                            float scale, const float *h0, void *o, float *hT,
                            const int *cu_seqlens, int N, int T_total, int Hk, int H, int dk,
                            int dv, const gla_headgate_layout *layout, void *, unsigned long,
                            cudaStream_t stream) {
    using namespace gla;
    if (!layout || !bounds_ok(cu_seqlens, N, T_total)) return GLA_ERR_ARG;
    if (T_total > 0 && (!q || !k || !v || !log_alpha || !o)) return GLA_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(h0) | reinterpret_cast<uintptr_t>(hT)) & 15) return GLA_ERR_ARG;
    int st = headgate_check(q, k, v, log_alpha, nullptr, o, Hk, H, dk, dv, *layout);
    if (st != GLA_OK) return st;
    if (T_total > 1 && (!layout->q_st || !layout->k_st || !layout->v_st)) return GLA_ERR_ARG;
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    TokenArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.log_alpha = log_alpha;
    a.h0 = h0;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.hT = hT;
    a.lay = *layout;
    a.scale = scale;
    a.H = H;
    a.share = H / Hk;
    a.dk = dk;
    a.dv = dv;
    for (a.first = 0; a.first < N; a.first += kBounds) {
        const int n = std::min(kBounds, N - a.first);
        std::copy(cu_seqlens + a.first, cu_seqlens + a.first + n + 1, a.bounds);
        headgate_token_kernel<<<dim3(H, (dv + kCols - 1) / kCols, n), kCols, 0, stream>>>(a);
        if (cudaGetLastError() != cudaSuccess) return GLA_ERR_LAUNCH;
    }
    return GLA_OK;
}

}  // extern "C"
