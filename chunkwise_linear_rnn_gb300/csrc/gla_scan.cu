// gla_scan.cu — the gated linear recurrence of one state value per channel,
//     h_t = exp(log_alpha_t) h_{t-1} + x_t,
// forward, backward, packed batches and the decode step.
//
// A thread block takes a tile of consecutive tokens and neighbouring channels in
// registers, its threads a few tokens each; each maps the state before its tokens to
// the state after them, and these maps are joined over the block and, where few
// sequences leave the device idle, over a cluster of blocks that stand side by side
// in time.  The blocks walk the sequence together, tile after tile.  No block waits
// for another but at its cluster's barrier, nothing is added in an order that the
// scheduler chooses, and no memory but the arguments is used.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>
#include <vector>

#include "gla.h"
#include "gla_internal.h"
#include "gla_ptx.cuh"

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
    int D, H, nseq, cluster;
    ScanSeq seqs[kMaxSeqs];
};

// The shape of one thread block: kThreads threads in runs of LPR lanes.  A run
// takes LPR * VEC neighbouring channels of TPW consecutive tokens, and the
// block's runs follow one another in time, so that its tile is
// (kThreads / LPR) * TPW tokens of LPR * VEC channels.
constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;

template <int VEC, int LPR, int TPW>
struct Tile {
    static constexpr int kChannels = LPR * VEC;
    static constexpr int kRuns = kThreads / LPR;
    static constexpr int kTokens = kRuns * TPW;
    static_assert(kBlock % TPW == 0 && 2 * kChannels <= kThreads, "tile");
};

// VEC neighbouring values as they lie in memory.
template <typename E, int VEC>
struct Raw;
template <>
struct Raw<float, 1> {
    float v;
    __device__ __forceinline__ float at(int) const { return v; }
};
template <>
struct Raw<float, 4> {
    float4 v;
    __device__ __forceinline__ float at(int i) const {
        return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ float at(int) const { return __bfloat162float(v); }
};
template <>
struct Raw<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ float at(int i) const {
        const unsigned w = i < 2 ? v.x : v.y;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};

template <typename E, int VEC>
__device__ __forceinline__ Raw<E, VEC> load(const void *p, size_t i) {
    return *reinterpret_cast<const Raw<E, VEC> *>(static_cast<const E *>(p) + i);
}

template <int VEC>
__device__ __forceinline__ void store(float *p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else p[0] = v[0];
}
template <int VEC>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const unsigned *>(&a),
                                                   *reinterpret_cast<const unsigned *>(&b));
    } else {
        p[0] = __float2bfloat16_rn(v[0]);
    }
}
template <int VEC>
__device__ __forceinline__ void fetch(const float *p, float (&v)[VEC]) {
    const Raw<float, VEC> r = *reinterpret_cast<const Raw<float, VEC> *>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r.at(i);
}

// Where a thread stands: its unit's (one sequence of one head, one group of
// channels) rows, states and checkpoints, and its own place in the tile.
struct Place {
    unsigned rank, cl;       // this block in its cluster, blocks of the cluster
    unsigned len;            // tokens of the sequence
    bool valid;              // its channels exist
    int first;               // first channel of the group
    size_t row, state, ck;   // elements: first row, state and checkpoint of its channels
};

template <int VEC, int LPR, int TPW>
__device__ __forceinline__ Place place(const ScanArgs &p) {
    using G = Tile<VEC, LPR, TPW>;
    Place o;
    o.cl = p.cluster;
    o.rank = blockIdx.x % p.cluster;
    const unsigned groups = (p.D + G::kChannels - 1) / G::kChannels;
    const unsigned work = blockIdx.x / p.cluster;
    const unsigned unit = work / groups;
    o.first = (work % groups) * G::kChannels;
    const int c = o.first + (threadIdx.x % LPR) * VEC;
    const unsigned head = unit % p.H;
    const ScanSeq s = p.seqs[unit / p.H];
    o.len = s.len;
    o.valid = c < p.D;
    o.row = (static_cast<size_t>(head) * p.rows + s.first) * p.D + c;
    o.state = (static_cast<size_t>(s.n) * p.H + head) * p.D + c;
    o.ck = (static_cast<size_t>(head) * p.blocks + s.block) * p.D + c;
    return o;
}

// Stores (a, b) as block `rank`'s entry of channel c in every block of the cluster.
template <int CH>
__device__ __forceinline__ void publish(float2 (*agg)[CH], unsigned rank, unsigned cl, int c,
                                        float a, float b) {
    if (cl == 1) {
        agg[0][c] = make_float2(a, b);
        return;
    }
    const uint32_t at = smem_u32(&agg[rank][c]);
    for (unsigned j = 0; j < cl; ++j)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(at, j)), "f"(a),
                     "f"(b)
                     : "memory");
}

__device__ __forceinline__ void sync_all(unsigned cl) {
    if (cl == 1) __syncthreads();
    else cluster_sync_all();
}

// Forward.  Per tile: each run reduces its tokens to the pair (P, H) that maps
// the state before them to the state after them, h -> P h + H; the runs' pairs
// are scanned in the block, the blocks' pairs exchanged in the cluster, and each
// run walks its tokens again from its true state, from registers.
template <typename E, int VEC, int LPR, int TPW>
__global__ void __launch_bounds__(kThreads, 3) scan_fwd_kernel(const __grid_constant__ ScanArgs p) {
    using G = Tile<VEC, LPR, TPW>;
    constexpr int CH = G::kChannels, RUNS = G::kRuns;
    __shared__ float2 s_run[RUNS][CH];
    // two of them: a block may publish its next tile while another still reads this one
    __shared__ float2 s_agg[2][kMaxCluster][CH];
    const int tid = threadIdx.x, run = tid / LPR, cl0 = (tid % LPR) * VEC;
    const Place o = place<VEC, LPR, TPW>(p);
    float carry[VEC] = {};
    if (p.h0 && o.valid) fetch<VEC>(p.h0 + o.state, carry);
    if (o.len == 0) {
        if (p.hT && o.valid && o.rank == 0 && run == 0) store<VEC>(p.hT + o.state, carry);
        return;
    }
    int buf = 0;
    for (unsigned base = 0; base < o.len; base += o.cl * G::kTokens, buf ^= 1) {
        const unsigned t0 = base + o.rank * G::kTokens + run * TPW;
        const size_t at = o.row + static_cast<size_t>(t0) * p.D;
        float a[TPW][VEC];
        Raw<E, VEC> x[TPW];
        Raw<float, VEC> l[TPW];
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
            x[i] = Raw<E, VEC>{};
            l[i] = Raw<float, VEC>{};   // a token past the end: gate 1, nothing written
            if (o.valid && t0 + i < o.len) {
                l[i] = load<float, VEC>(p.log_alpha, at + static_cast<size_t>(i) * p.D);
                x[i] = load<E, VEC>(p.x, at + static_cast<size_t>(i) * p.D);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float P = 1.f, H = 0.f;
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
                a[i][v] = expf(l[i].at(v));
                H = fmaf(a[i][v], H, x[i].at(v));
                P *= a[i][v];
            }
            s_run[run][cl0 + v] = make_float2(P, H);
        }
        __syncthreads();
        if (tid < CH) {
            float P = 1.f, H = 0.f;
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                const float2 q = s_run[r][tid];
                s_run[r][tid] = make_float2(P, H);
                H = fmaf(q.x, H, q.y);
                P *= q.x;
            }
            publish<CH>(s_agg[buf], o.rank, o.cl, tid, P, H);
        }
        sync_all(o.cl);
        float h[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = carry[v];
        for (unsigned j = 0; j < o.cl; ++j) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (j == o.rank) h[v] = carry[v];
                const float2 q = s_agg[buf][j][cl0 + v];
                carry[v] = fmaf(q.x, carry[v], q.y);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float2 q = s_run[run][cl0 + v];
            h[v] = fmaf(q.x, h[v], q.y);
        }
        if (o.valid && t0 < o.len) {
            if (p.ckpt_out && t0 % kBlock == 0)
                store<VEC>(p.ckpt_out + o.ck + static_cast<size_t>(t0 / kBlock) * p.D, h);
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = fmaf(a[i][v], h[v], x[i].at(v));
                if (p.h && t0 + i < o.len)
                    store<VEC>(static_cast<E *>(p.h) + at + static_cast<size_t>(i) * p.D, h);
            }
            if (p.hT && o.len - t0 <= TPW) store<VEC>(p.hT + o.state, h);
        }
    }
}

// Backward, from the last tile to the first.  Forward in time, the states
// h_{t-1} are walked again from the checkpoint of each block of kBlock tokens;
// backward in time, u_t = alpha_t g_t is the recurrence's own scan from the end:
// a run maps the u that enters it on the right to the one that leaves it on the
// left, u -> P u + U, with the same P.  Products and sums are rounded one by one,
// so that a call with fewer outputs gives the same bits.
template <typename E, int VEC, int LPR, int TPW>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const __grid_constant__ ScanArgs p) {
    using G = Tile<VEC, LPR, TPW>;
    constexpr int CH = G::kChannels, RUNS = G::kRuns, RPB = kBlock / TPW;   // runs of a block
    static_assert(RUNS % RPB == 0, "a tile is whole blocks");
    __shared__ float s_p[RUNS][CH];
    __shared__ float s_h[RUNS][CH];   // a run's H, then the state that enters it
    __shared__ float s_u[RUNS][CH];   // a run's U, then that of the runs to its right
    __shared__ float s_q[RUNS][CH];   // the P of the runs to its right
    __shared__ float2 s_agg[2][kMaxCluster][CH];
    const int tid = threadIdx.x, run = tid / LPR, cl0 = (tid % LPR) * VEC;
    const Place o = place<VEC, LPR, TPW>(p);
    float carry[VEC] = {};
    if (p.dhT && o.valid) fetch<VEC>(p.dhT + o.state, carry);
    if (o.len == 0) {
        if (p.hT && o.valid && o.rank == 0 && run == 0) store<VEC>(p.hT + o.state, carry);
        return;
    }
    // the channel that this thread scans over the runs: the first CH threads forward,
    // the next CH backward
    const int sc = tid % CH;
    const size_t sck = o.ck - cl0 + sc;
    const bool svalid = tid < CH && o.first + sc < p.D;
    const unsigned span = o.cl * G::kTokens;
    int buf = 0;
    for (unsigned left = (o.len - 1) / span + 1; left-- > 0; buf ^= 1) {
        const unsigned tile0 = left * span + o.rank * G::kTokens;
        const unsigned t0 = tile0 + run * TPW;
        const size_t at = o.row + static_cast<size_t>(t0) * p.D;
        float a[TPW][VEC];
        Raw<E, VEC> x[TPW], d[TPW];
        {
            Raw<float, VEC> l[TPW];
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
                x[i] = d[i] = Raw<E, VEC>{};
                l[i] = Raw<float, VEC>{};   // a token past the end: gate 1, nothing written
                if (o.valid && t0 + i < o.len) {
                    l[i] = load<float, VEC>(p.log_alpha, at + static_cast<size_t>(i) * p.D);
                    x[i] = load<E, VEC>(p.x, at + static_cast<size_t>(i) * p.D);
                    if (p.d_h) d[i] = load<E, VEC>(p.d_h, at + static_cast<size_t>(i) * p.D);
                }
            }
            float P[VEC], H[VEC], U[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                P[v] = 1.f, H[v] = 0.f, U[v] = 0.f;
#pragma unroll
                for (int i = 0; i < TPW; ++i) {
                    a[i][v] = expf(l[i].at(v));
                    H[v] = fmaf(a[i][v], H[v], x[i].at(v));
                    P[v] *= a[i][v];
                }
#pragma unroll
                for (int i = TPW - 1; i >= 0; --i)
                    U[v] = __fmul_rn(a[i][v], __fadd_rn(U[v], d[i].at(v)));
            }
            store<VEC>(&s_p[run][cl0], P);
            store<VEC>(&s_h[run][cl0], H);
            store<VEC>(&s_u[run][cl0], U);
        }
        float ck[RUNS / RPB];
#pragma unroll
        for (int b = 0; b < RUNS / RPB; ++b) {
            const unsigned t = tile0 + b * kBlock;
            ck[b] = svalid && t < o.len
                        ? p.ckpt_in[sck + static_cast<size_t>(t / kBlock) * p.D] : 0.f;
        }
        __syncthreads();
        if (tid < CH) {
            float h = 0.f;
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                if (r % RPB == 0) h = ck[r / RPB];
                const float H = s_h[r][sc];
                s_h[r][sc] = h;
                h = fmaf(s_p[r][sc], h, H);
            }
        } else if (tid < 2 * CH) {
            float P = 1.f, U = 0.f;
#pragma unroll
            for (int r = RUNS - 1; r >= 0; --r) {
                const float q = s_p[r][sc], w = s_u[r][sc];
                s_u[r][sc] = U;
                s_q[r][sc] = P;
                U = fmaf(q, U, w);
                P *= q;
            }
            publish<CH>(s_agg[buf], o.rank, o.cl, sc, P, U);
        }
        sync_all(o.cl);
        float u[VEC], h[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) u[v] = carry[v];
        for (unsigned j = o.cl; j-- > 0;) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (j == o.rank) u[v] = carry[v];
                const float2 q = s_agg[buf][j][cl0 + v];
                carry[v] = fmaf(q.x, carry[v], q.y);
            }
        }
        float q[VEC], w[VEC];
        fetch<VEC>(&s_q[run][cl0], q);
        fetch<VEC>(&s_u[run][cl0], w);
        fetch<VEC>(&s_h[run][cl0], h);
#pragma unroll
        for (int v = 0; v < VEC; ++v) u[v] = fmaf(q[v], u[v], w[v]);
        if (o.valid && t0 < o.len) {
            float before[TPW][VEC];
#pragma unroll
            for (int i = 0; i < TPW; ++i)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    before[i][v] = h[v];
                    h[v] = fmaf(a[i][v], h[v], x[i].at(v));
                }
#pragma unroll
            for (int i = TPW - 1; i >= 0; --i) {
                float g[VEC], da[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    g[v] = __fadd_rn(u[v], d[i].at(v));
                    u[v] = __fmul_rn(a[i][v], g[v]);
                    da[v] = __fmul_rn(u[v], before[i][v]);
                }
                if (t0 + i < o.len) {
                    const size_t e = at + static_cast<size_t>(i) * p.D;
                    if (p.h) store<VEC>(static_cast<E *>(p.h) + e, g);
                    if (p.ga) store<VEC>(p.ga + e, da);
                }
            }
            if (p.hT && t0 == 0) store<VEC>(p.hT + o.state, u);
        }
    }
}

// The decode step: VEC values a thread, one pass over the state.
template <typename E, int VEC>
__global__ void __launch_bounds__(256)
    scan_step_kernel(const E *x, const float *log_alpha, float *h, E *out, long long n) {
    const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * VEC;
    if (i >= n) return;
    const Raw<E, VEC> xv = load<E, VEC>(x, i);
    float s[VEC], l[VEC];
    fetch<VEC>(log_alpha + i, l);
    fetch<VEC>(h + i, s);
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = fmaf(expf(l[v]), s[v], xv.at(v));
    store<VEC>(h + i, s);
    store<VEC>(out + i, s);
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
    // thread blocks of the narrowest tiles in the longest clusters
    if (states * ((D + 31) / 32) > 0x7fffffffLL / kMaxCluster) return GLA_ERR_ARG;
    return GLA_OK;
}

template <typename E, int VEC, int LPR, int TPW>
int launch(ScanArgs &a, bool backward, int cluster, cudaStream_t stream) {
    constexpr int CH = Tile<VEC, LPR, TPW>::kChannels;
    const long long units = static_cast<long long>(a.nseq) * a.H * ((a.D + CH - 1) / CH);
    a.cluster = cluster;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    const ScanArgs &args = a;
    return static_cast<int>(backward
                                ? cudaLaunchKernelEx(&cfg, scan_bwd_kernel<E, VEC, LPR, TPW>, args)
                                : cudaLaunchKernelEx(&cfg, scan_fwd_kernel<E, VEC, LPR, TPW>, args));
}

// Lanes of a run (channels of a thread block / VEC) and blocks of a cluster for one launch.
struct Plan {
    int lpr, cluster;
};

Plan plan_of(const ScanArgs &a, int vec, int longest, int sms) {
    Plan best{32, 1};
    const long long slots = 3LL * sms;
    const long long units = static_cast<long long>(a.nseq) * a.H;
    // narrower tiles, then longer clusters, until the blocks fill the device once
    for (int lpr = 32; lpr >= (vec == 4 ? 8 : 32); lpr /= 2) {
        best.lpr = lpr;
        const long long u = units * ((a.D + lpr * vec - 1) / (lpr * vec));
        const long long tiles = (longest + (256 / lpr) * 8 - 1) / ((256 / lpr) * 8);
        best.cluster = 1;
        while (best.cluster < kMaxCluster && u * best.cluster * 2 <= slots &&
               best.cluster * 2 <= tiles)
            best.cluster *= 2;
        if (u * best.cluster * 2 > slots) break;
    }
    return best;
}

template <typename E>
int launch_for(ScanArgs &a, bool backward, bool vec4, const Plan &pl, cudaStream_t stream) {
    if (!vec4) return launch<E, 1, 32, 8>(a, backward, pl.cluster, stream);
    if (pl.lpr == 32) return launch<E, 4, 32, 8>(a, backward, pl.cluster, stream);
    if (pl.lpr == 16) return launch<E, 4, 16, 8>(a, backward, pl.cluster, stream);
    return launch<E, 4, 8, 8>(a, backward, pl.cluster, stream);
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
    const bool vec4 = D % 4 == 0 && aligned(16, a.x, a.log_alpha, a.h0, a.dhT, a.ckpt_in, a.d_h, a.h,
                                            a.hT, a.ga, a.ckpt_out);
    // longest first, so that the last thread blocks to start are short ones
    std::stable_sort(seqs.begin(), seqs.end(),
                     [](const ScanSeq &x, const ScanSeq &y) { return x.len > y.len; });
    for (int n = 0; n < N; n += kMaxSeqs) {
        a.nseq = std::min(kMaxSeqs, N - n);
        std::copy(seqs.begin() + n, seqs.begin() + n + a.nseq, a.seqs);
        const Plan pl = plan_of(a, vec4 ? 4 : 1, seqs[n].len, sms);
        const int e = dtype == GLA_BF16 ? launch_for<__nv_bfloat16>(a, backward, vec4, pl, stream)
                                        : launch_for<float>(a, backward, vec4, pl, stream);
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
    const bool vec4 = n % 4 == 0 && aligned(16, x, log_alpha, h, out);
    const long long blocks = (n + (vec4 ? 1023 : 255)) / (vec4 ? 1024 : 256);
    if (blocks > 0x7fffffffLL) return GLA_ERR_ARG;
    int sms = 0;
    const int st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const unsigned grid = static_cast<unsigned>(blocks);
    const auto go = [&](auto kernel, auto *xe) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(xe)>>;
        kernel<<<grid, 256, 0, stream>>>(xe, log_alpha, h, static_cast<E *>(out), n);
    };
    if (dtype == GLA_BF16) {
        const auto *xe = static_cast<const __nv_bfloat16 *>(x);
        if (vec4) go(scan_step_kernel<__nv_bfloat16, 4>, xe);
        else go(scan_step_kernel<__nv_bfloat16, 1>, xe);
    } else {
        const auto *xe = static_cast<const float *>(x);
        if (vec4) go(scan_step_kernel<float, 4>, xe);
        else go(scan_step_kernel<float, 1>, xe);
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // extern "C"
