// gla_scan.cu — the gated linear recurrence of one state value per channel,
//     h_t = exp(log_alpha_t) h_{t-1} + x_t,
// forward, backward, packed batches and the decode step.
//
// One thread walks one channel of one sequence, token after token; the 32
// channels of a warp are neighbours, so that every load and store of a token is
// one contiguous run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "gla.h"
#include "gla_internal.h"

namespace gla {
namespace {

constexpr int kBlock = GLA_SCAN_BLOCK;
constexpr int kMaxSeqs = 200;   // sequences of one launch: their table travels as a parameter

// One sequence: its rows [first, first + len) of every head, its number n in
// the caller's order and its first block of checkpoints.
struct ScanSeq {
    int first, len, n, block;
};

struct ScanArgs {
    const void *x;
    const float *log_alpha;
    const float *h0, *dhT;
    const float *ckpt_in;
    const void *d_h;
    void *h;                 // forward: h; backward: grad_x
    float *hT;               // forward: hT; backward: grad_h0
    float *ga;
    float *ckpt_out;
    long long rows;          // rows of one head
    long long blocks;        // checkpoint blocks of one head
    int D, H, nseq;
    ScanSeq seqs[kMaxSeqs];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <typename E>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const __grid_constant__ ScanArgs p) {
    const int groups = (p.D + 127) / 128;
    const int unit = blockIdx.x / groups;
    const int c = (blockIdx.x % groups) * 128 + threadIdx.x;
    if (c >= p.D) return;
    const int head = unit % p.H;
    const ScanSeq s = p.seqs[unit / p.H];
    const size_t at = (static_cast<size_t>(head) * p.rows + s.first) * p.D + c;
    const size_t state = (static_cast<size_t>(s.n) * p.H + head) * p.D + c;
    const size_t ck = (static_cast<size_t>(head) * p.blocks + s.block) * p.D + c;
    float h = p.h0 ? p.h0[state] : 0.f;
    for (int t = 0; t < s.len; ++t) {
        if (p.ckpt_out && t % kBlock == 0) p.ckpt_out[ck + static_cast<size_t>(t / kBlock) * p.D] = h;
        const size_t i = at + static_cast<size_t>(t) * p.D;
        h = fmaf(expf(p.log_alpha[i]), h, to_f32(static_cast<const E *>(p.x)[i]));
        if (p.h) put(static_cast<E *>(p.h) + i, h);
    }
    if (p.hT) p.hT[state] = h;
}

template <typename E>
__global__ void __launch_bounds__(128) scan_bwd_kernel(const __grid_constant__ ScanArgs p) {
    const int groups = (p.D + 127) / 128;
    const int unit = blockIdx.x / groups;
    const int c = (blockIdx.x % groups) * 128 + threadIdx.x;
    if (c >= p.D) return;
    const int head = unit % p.H;
    const ScanSeq s = p.seqs[unit / p.H];
    const size_t at = (static_cast<size_t>(head) * p.rows + s.first) * p.D + c;
    const size_t state = (static_cast<size_t>(s.n) * p.H + head) * p.D + c;
    const size_t ck = (static_cast<size_t>(head) * p.blocks + s.block) * p.D + c;
    float u = p.dhT ? p.dhT[state] : 0.f;
    for (int b = (s.len + kBlock - 1) / kBlock - 1; b >= 0; --b) {
        const int t0 = b * kBlock, n = min(kBlock, s.len - t0);
        float before[kBlock];
        float h = p.ckpt_in[ck + static_cast<size_t>(b) * p.D];
        for (int j = 0; j < n; ++j) {
            const size_t i = at + static_cast<size_t>(t0 + j) * p.D;
            before[j] = h;
            h = fmaf(expf(p.log_alpha[i]), h, to_f32(static_cast<const E *>(p.x)[i]));
        }
        for (int j = n - 1; j >= 0; --j) {
            const size_t i = at + static_cast<size_t>(t0 + j) * p.D;
            // each product and sum rounded by itself, so that the same call with fewer
            // outputs gives the same bits
            const float g = __fadd_rn(u, p.d_h ? to_f32(static_cast<const E *>(p.d_h)[i]) : 0.f);
            u = __fmul_rn(expf(p.log_alpha[i]), g);
            if (p.h) put(static_cast<E *>(p.h) + i, g);
            if (p.ga) p.ga[i] = __fmul_rn(u, before[j]);
        }
    }
    if (p.hT) p.hT[state] = u;
}

template <typename E>
__global__ void __launch_bounds__(256)
    scan_step_kernel(const E *x, const float *log_alpha, float *h, E *out, long long n) {
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const float v = fmaf(expf(log_alpha[i]), h[i], to_f32(x[i]));
    h[i] = v;
    put(out + i, v);
}

// Whether every address is a multiple of `n` bytes (a null pointer is).
template <typename... P>
bool aligned(unsigned n, P... p) {
    return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t{0}) & (n - 1)) == 0;
}

bool elements_aligned(const ScanArgs &a, int dtype) {
    return aligned(dtype == GLA_BF16 ? 2 : 4, a.x, a.d_h, a.h) &&
           aligned(4, a.log_alpha, a.h0, a.dhT, a.ckpt_in, a.hT, a.ga, a.ckpt_out);
}

// Checks shared by the scans; cu_seqlens [N + 1] is checked by the caller's loop.
int check_common(const ScanArgs &a, long long states, int D, int dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_ARG;
    if (!elements_aligned(a, dtype)) return GLA_ERR_ARG;
    if (states * ((D + 127) / 128) > 0x7fffffffLL) return GLA_ERR_ARG;
    return GLA_OK;
}

template <typename E>
int launch(const ScanArgs &a, bool backward, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.nseq) * a.H *
                                                ((a.D + 127) / 128));
    if (backward) scan_bwd_kernel<E><<<grid, 128, 0, stream>>>(a);
    else scan_fwd_kernel<E><<<grid, 128, 0, stream>>>(a);
    return static_cast<int>(cudaGetLastError());
}

// Forward or backward over N sequences of H heads (a fixed-length batch is one
// sequence of B heads).
int run(ScanArgs &a, bool backward, const int *cu_seqlens, int N, int H, int T_total, int D,
        int dtype, cudaStream_t stream) {
    if (!cu_seqlens || N <= 0 || H <= 0 || T_total < 0 || D <= 0) return GLA_ERR_ARG;
    int st = check_common(a, static_cast<long long>(N) * H, D, dtype);
    if (st != GLA_OK) return st;
    if (cu_seqlens[0] != 0 || cu_seqlens[N] != T_total) return GLA_ERR_ARG;
    std::vector<ScanSeq> seqs(N);
    long long blocks = 0;
    for (int n = 0; n < N; ++n) {
        const long long len = static_cast<long long>(cu_seqlens[n + 1]) - cu_seqlens[n];
        if (len < 0) return GLA_ERR_ARG;
        seqs[n] = ScanSeq{cu_seqlens[n], static_cast<int>(len), n, static_cast<int>(blocks)};
        blocks += (len + kBlock - 1) / kBlock;
    }
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    a.rows = T_total;
    a.blocks = blocks;
    a.D = D;
    a.H = H;
    // longest first, so that the last thread blocks to start are short ones
    std::stable_sort(seqs.begin(), seqs.end(),
                     [](const ScanSeq &x, const ScanSeq &y) { return x.len > y.len; });
    for (int n = 0; n < N; n += kMaxSeqs) {
        a.nseq = std::min(kMaxSeqs, N - n);
        std::copy(seqs.begin() + n, seqs.begin() + n + a.nseq, a.seqs);
        const int e = dtype == GLA_BF16 ? launch<__nv_bfloat16>(a, backward, stream)
                                        : launch<float>(a, backward, stream);
        if (e != 0) return GLA_ERR_LAUNCH;
    }
    return GLA_OK;
}

}  // namespace
}  // namespace gla

extern "C" {

int gla_scan_fwd_varlen(const void *x, const float *log_alpha, const float *h0, void *h,
                        float *hT, float *checkpoints, const int *cu_seqlens, int N, int H,
                        int T_total, int D, int dtype, cudaStream_t stream) {
    // a packed batch of empty sequences has no rows to point at
    if (T_total > 0 && (!x || !log_alpha || (!h && !hT && !checkpoints))) return GLA_ERR_ARG;
    gla::ScanArgs a = {};
    a.x = x;
    a.log_alpha = log_alpha;
    a.h0 = h0;
    a.h = h;
    a.hT = hT;
    a.ckpt_out = checkpoints;
    return gla::run(a, false, cu_seqlens, N, H, T_total, D, dtype, stream);
}

int gla_scan_fwd(const void *x, const float *log_alpha, const float *h0, void *h, float *hT,
                 float *checkpoints, int B, int T, int D, int dtype, cudaStream_t stream) {
    if (T <= 0) return GLA_ERR_ARG;
    const int cu[2] = {0, T};
    return gla_scan_fwd_varlen(x, log_alpha, h0, h, hT, checkpoints, cu, 1, B, T, D, dtype,
                               stream);
}

int gla_scan_bwd_varlen(const void *x, const float *log_alpha, const float *checkpoints,
                        const void *d_h, const float *dhT, void *grad_x, float *grad_log_alpha,
                        float *grad_h0, const int *cu_seqlens, int N, int H, int T_total, int D,
                        int dtype, cudaStream_t stream) {
    if (T_total > 0 &&
        (!x || !log_alpha || !checkpoints || (!grad_x && !grad_log_alpha && !grad_h0)))
        return GLA_ERR_ARG;
    gla::ScanArgs a = {};
    a.x = x;
    a.log_alpha = log_alpha;
    a.ckpt_in = checkpoints;
    a.d_h = d_h;
    a.dhT = dhT;
    a.h = grad_x;
    a.ga = grad_log_alpha;
    a.hT = grad_h0;
    return gla::run(a, true, cu_seqlens, N, H, T_total, D, dtype, stream);
}

int gla_scan_bwd(const void *x, const float *log_alpha, const float *checkpoints, const void *d_h,
                 const float *dhT, void *grad_x, float *grad_log_alpha, float *grad_h0, int B,
                 int T, int D, int dtype, cudaStream_t stream) {
    if (T <= 0) return GLA_ERR_ARG;
    const int cu[2] = {0, T};
    return gla_scan_bwd_varlen(x, log_alpha, checkpoints, d_h, dhT, grad_x, grad_log_alpha,
                               grad_h0, cu, 1, B, T, D, dtype, stream);
}

int gla_scan_step(const void *x, const float *log_alpha, float *h, void *out, int B, int D,
                  int dtype, cudaStream_t stream) {
    using namespace gla;
    if (!x || !log_alpha || !h || !out || B <= 0 || D <= 0) return GLA_ERR_ARG;
    if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_ARG;
    if (!aligned(dtype == GLA_BF16 ? 2 : 4, x, out) || !aligned(4, log_alpha, h)) return GLA_ERR_ARG;
    const long long n = static_cast<long long>(B) * D;
    if ((n + 255) / 256 > 0x7fffffffLL) return GLA_ERR_ARG;
    int sms = 0;
    const int st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const unsigned grid = static_cast<unsigned>((n + 255) / 256);
    if (dtype == GLA_BF16)
        scan_step_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16 *>(x), log_alpha,
                                                   h, static_cast<__nv_bfloat16 *>(out), n);
    else
        scan_step_kernel<<<grid, 256, 0, stream>>>(static_cast<const float *>(x), log_alpha, h,
                                                   static_cast<float *>(out), n);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // extern "C"
