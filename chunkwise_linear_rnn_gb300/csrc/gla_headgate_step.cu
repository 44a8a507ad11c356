// gla_headgate_step.cu — one token of the recurrence with one gate per head, for states that
// lie in a pool:
//     h <- a h + k^T v,     o = scale q h   (updated h),   a = exp(log_alpha)
// per row and value head, q and k of the key head that it shares.
//
// A stream of the fp32 state: 8 dk dv bytes a head against 5 dk dv operations, bound by HBM.  A
// block takes one head's columns (or a tile of them); a thread owns one 16-byte column group of
// up to 16 rows, all of whose loads are issued before any use.  The sum over the rows runs in
// registers, over the lanes that share columns by shuffles, and over warps in shared memory.
// Measured on one GB300: 256 rows of 32 heads of 128 x 128 157 us (6.9 TB/s, a copy's 6.79);
// 4 rows of 16 heads 3.2 us, which is latency (slot, then state, then the sums).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "gla.h"
#include "gla_exp.cuh"
#include "gla_internal.h"
#include "gla_ptx.cuh"

namespace gla {
namespace {

struct StepArgs {
    const void *q, *k, *v;
    const float *log_alpha;
    const long long *slots;
    float *h;
    void *o;
    gla_headgate_layout lay;
    float scale;
    int S, H, share, dk, dv;     // share: value heads of a key head
    unsigned int *status;
};

__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(float x) { return x; }

__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

constexpr int kMaxDk = 128;

// G column groups of 4: a tile of 4 G columns, and as many threads as leave each at most 16 of
// up to 128 rows.
template <int G>
struct Tile {
    static constexpr int kThreads = G == 64 ? 512 : 256;
    static constexpr int kRowBases = kThreads / G;
    static constexpr int kRows = kMaxDk / kRowBases;
    static constexpr int kWarps = kThreads / 32;
};

template <typename E, int G>
__global__ void __launch_bounds__(Tile<G>::kThreads) headgate_step_kernel(const StepArgs p) {
    using L = Tile<G>;
    constexpr int RB = L::kRowBases;
    __shared__ float s_q[kMaxDk], s_k[kMaxDk];
    __shared__ float4 s_red[L::kWarps][G < 32 ? G : 32];
    const int tid = threadIdx.x, cg = tid % G, rb = tid / G;
    const int head = blockIdx.x % p.H, b = blockIdx.x / p.H, hk = head / p.share;
    const int c = (blockIdx.y * G + cg) * 4;
    const bool mine = c < p.dv;
    const long long slot = p.slots ? p.slots[b] : b;
    const bool real = slot >= 0 && slot < p.S;

    float4 *hs = reinterpret_cast<float4 *>(
        p.h + ((real ? slot : 0) * p.H + head) * static_cast<long long>(p.dk) * p.dv + c);
    const long long row4 = p.dv / 4;
    float4 s[L::kRows];
#pragma unroll
    for (int m = 0; m < L::kRows; ++m) {
        const int d = rb + m * RB;
        s[m] = real && mine && d < p.dk ? __ldcs(hs + d * row4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < p.dk) {
        s_q[tid] = widen(static_cast<const E *>(p.q)[b * p.lay.q_st + hk * p.lay.q_sh + tid]);
        s_k[tid] = widen(static_cast<const E *>(p.k)[b * p.lay.k_st + hk * p.lay.k_sh + tid]);
    }
    const float a = exp_centred(p.log_alpha[b * p.lay.a_st + head * p.lay.a_sh]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine) v = load4(static_cast<const E *>(p.v) + b * p.lay.v_st + head * p.lay.v_sh + c);
    // the state belongs to the first row that names it
    bool taken = false;
    if (p.slots && real)
        for (int i = tid; i < b; i += L::kThreads) taken = taken || p.slots[i] == slot;
    taken = __syncthreads_or(taken) != 0;
    const bool use = real && !taken;
    if (tid == 0 && slot >= 0 && !use) atomicOr(p.status, kStatusSlot);

    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < L::kRows; ++m) {
        const int d = rb + m * RB;
        if (!use || !mine || d >= p.dk) continue;
        const float kd = s_k[d], qd = s_q[d];
        float4 t = s[m];
        t.x = fmaf(a, t.x, kd * v.x);
        t.y = fmaf(a, t.y, kd * v.y);
        t.z = fmaf(a, t.z, kd * v.z);
        t.w = fmaf(a, t.w, kd * v.w);
        __stcs(hs + d * row4, t);
        acc.x = fmaf(qd, t.x, acc.x);
        acc.y = fmaf(qd, t.y, acc.y);
        acc.z = fmaf(qd, t.z, acc.z);
        acc.w = fmaf(qd, t.w, acc.w);
    }

    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int off = G; off < 32; off <<= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
    }
    if (G >= 32 || lane < G) s_red[warp][lane] = acc;
    __syncthreads();
    if (tid < G && mine) {
        // warps per set of 32 column groups
        constexpr int W = G < 32 ? 1 : G / 32;
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < L::kWarps / W; ++w) {
            const float4 x = s_red[w * W + tid / 32][tid % 32];
            r.x += x.x;
            r.y += x.y;
            r.z += x.z;
            r.w += x.w;
        }
        // a row of padding gives zeros, whatever its q holds
        E *o = static_cast<E *>(p.o) + (static_cast<long long>(b) * p.H + head) * p.dv + c;
        store4(o, use ? make_float4(p.scale * r.x, p.scale * r.y, p.scale * r.z, p.scale * r.w)
                      : make_float4(0.f, 0.f, 0.f, 0.f));
    }
}

template <typename E, int G>
int launch_tile(const StepArgs &a, unsigned heads, cudaStream_t stream) {
    const dim3 grid(heads, (a.dv / 4 + G - 1) / G);
    headgate_step_kernel<E, G><<<grid, Tile<G>::kThreads, 0, stream>>>(a);
    return static_cast<int>(cudaGetLastError());
}

template <typename E>
int launch(const StepArgs &a, unsigned heads, int sms, cudaStream_t stream) {
    // The narrowest tile that holds the columns; where heads are fewer than two for each SM, tiles
    // of 32 columns, so that more SMs have a part of them (4 rows of 16 heads of 128 x 128: 3.2 us,
    // 3.7 with whole rows; 256 rows of 32 heads: 157 us whole, 167 in tiles of 32).
    if (a.dv <= 32 || heads < 2u * sms) return launch_tile<E, 8>(a, heads, stream);
    if (a.dv <= 64) return launch_tile<E, 16>(a, heads, stream);
    if (a.dv <= 128) return launch_tile<E, 32>(a, heads, stream);
    return launch_tile<E, 64>(a, heads, stream);
}

}  // namespace
}  // namespace gla

extern "C" int gla_headgate_step(const void *q, const void *k, const void *v,
                                 const float *log_alpha, float scale, float *h,
                                 const long long *slots, void *o, int B, int S, int Hk, int H,
                                 int dk, int dv, const gla_headgate_layout *layout, int dtype,
                                 cudaStream_t stream) {
    using namespace gla;
    if (!q || !k || !v || !log_alpha || !h || !o || !layout) return GLA_ERR_ARG;
    if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_ARG;
    if (B <= 0 || S <= 0 || (!slots && S < B)) return GLA_ERR_ARG;
    const int st = headgate_check(q, k, v, log_alpha, h, o, Hk, H, dk, dv, *layout);
    if (st != GLA_OK) return st;
    if ((reinterpret_cast<uintptr_t>(h) & 15) || (reinterpret_cast<uintptr_t>(slots) & 7))
        return GLA_ERR_ARG;
    if (static_cast<long long>(B) * H > INT_MAX) return GLA_ERR_ARG;
    const int size = dtype == GLA_BF16 ? 2 : 4;
    Span in[4];
    headgate_inputs(in, q, k, v, log_alpha, B, Hk, H, dk, dv, size, *layout);
    const Span pool = span_of(h, static_cast<unsigned long long>(S) * H * dk * dv, 4);
    const Span out = span_of(o, static_cast<unsigned long long>(B) * H * dv, size);
    const Span names = span_of(slots, B, 8);
    if (meets_any(pool, in) || meets_any(out, in) || meet(pool, out) || meet(pool, names) ||
        meet(out, names))
        return GLA_ERR_ARG;
    StepArgs a = {};
    int sms = 0;
    const int dev = usable_device(&sms, &a.status);
    if (dev != GLA_OK) return dev;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_alpha = log_alpha;
    a.slots = slots;
    a.h = h;
    a.o = o;
    a.lay = *layout;
    a.scale = scale;
    a.S = S;
    a.H = H;
    a.share = H / Hk;
    a.dk = dk;
    a.dv = dv;
    const unsigned heads = static_cast<unsigned>(B) * H;
    const int e = dtype == GLA_BF16 ? launch<__nv_bfloat16>(a, heads, sms, stream)
                                    : launch<float>(a, heads, sms, stream);
    return e == 0 ? GLA_OK : GLA_ERR_LAUNCH;
}
