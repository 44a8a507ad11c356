// gla_scan.cu — the gated linear recurrence of one state value per channel,
//     h_t = exp(log_alpha_t) h_{t-1} + x_t,
// forward, backward, packed batches and the decode step.
//
// A thread block takes a tile of consecutive tokens and neighbouring channels in
// registers, its threads a few tokens each; each maps the state before its tokens to
// the state after them, and these maps are joined over the block and, where few
// sequences leave the device idle, over a cluster of blocks that stand side by side
// in time.  The blocks walk the sequence together, tile after tile.  (A state that crosses
// tokens as P s loses what is left of it once P falls below fp32's range, 2^-126 of its size;
// a thread's own tokens and the decode step multiply gate by gate.)  A block waits for
// others of its own cluster only (and never longer than the library's limit), nothing is
// added in an order that the scheduler chooses, and no memory but the arguments is used.
//
// Short sequences in numbers take neither tiles nor exchange: a thread walks its own.
//
// Both directions are bound by HBM: 8 bytes an element forward (bf16 x, fp32 gates, bf16
// h), 14 backward, against about 20 instructions.  Measured on one GB300: forward B8 T2048
// D2048 42 us (6.3 TB/s of a copy's 6.67), B1 T262144 D1024 335 us (6.4 TB/s); backward B8
// T2048 D2048 80 us (5.9 TB/s).  With few sequences the blocks of one SM, not HBM, set the
// pace: two of them on some SMs and one on others.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <new>
#include <type_traits>
#include <vector>

#include "gla.h"
#include "gla_internal.h"
#include "gla_ptx.cuh"
#include "gla_scan_plan.h"

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
    CUtensorMap map_l, map_x, map_d;   // (channel, row, head), where TMA loads the tiles
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
    int cluster, width;      // thread blocks side by side in time, channels of a block
    unsigned int *status;    // device status word (bounded waits)
    ScanSeq seqs[kMaxSeqs];
};

// The shape of one thread block: kThreads threads in runs of LPR lanes.  A run
// takes LPR * VEC neighbouring channels of TPW consecutive tokens, and the
// block's runs follow one another in time, so that its tile is
// (kThreads / LPR) * TPW tokens of LPR * VEC channels.
template <int VEC, int LPR, int TPW, int THREADS>
struct Tile {
    static constexpr int kThreads = THREADS;
    static constexpr int kChannels = LPR * VEC;
    static constexpr int kRuns = kThreads / LPR;
    static constexpr int kTokens = kRuns * TPW;
    static_assert(kBlock % TPW == 0 && kChannels <= kThreads, "tile");
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
    unsigned start;          // its first row of the head
    int head;
    bool valid;              // its channels exist
    int first;               // first channel of the group
    size_t row, state, ck;   // elements: first row, state and checkpoint of its channels
};

template <typename G, int VEC, int LPR>
__device__ __forceinline__ Place place(const ScanArgs &p) {
    Place o;
    o.cl = cluster_of(G::kChannels) > 1 ? p.cluster : 1;
    o.rank = blockIdx.x % o.cl;
    const unsigned groups = (p.D + G::kChannels - 1) / G::kChannels;
    const unsigned work = blockIdx.x / o.cl;
    const unsigned unit = work / groups;
    o.first = (work % groups) * G::kChannels;
    const int c = o.first + (threadIdx.x % LPR) * VEC;
    const unsigned head = unit % p.H;
    const ScanSeq s = p.seqs[unit / p.H];
    o.len = s.len;
    o.start = s.first;
    o.head = head;
    o.valid = c < p.D;
    o.row = (static_cast<size_t>(head) * p.rows + s.first) * p.D + c;
    o.state = (static_cast<size_t>(s.n) * p.H + head) * p.D + c;
    o.ck = (static_cast<size_t>(head) * p.blocks + s.block) * p.D + c;
    return o;
}

// ---------------------------------------------------------------- arithmetic on VEC values

// Two fp32 operations in one instruction (each rounded as by itself).
__device__ __forceinline__ unsigned long long pair_of(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(unsigned long long r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// VEC fp32 values: a number, or two pairs.
template <int VEC>
struct Vec;
template <>
struct Vec<1> {
    float v;
    __device__ __forceinline__ static Vec all(float x) { return {x}; }
    __device__ __forceinline__ static Vec of(const float (&x)[1]) { return {x[0]}; }
    __device__ __forceinline__ void to(float (&x)[1]) const { x[0] = v; }
};
template <>
struct Vec<4> {
    unsigned long long lo, hi;
    __device__ __forceinline__ static Vec all(float x) { return {pair_of(x, x), pair_of(x, x)}; }
    __device__ __forceinline__ static Vec of(const float (&x)[4]) {
        return {pair_of(x[0], x[1]), pair_of(x[2], x[3])};
    }
    __device__ __forceinline__ void to(float (&x)[4]) const {
        unpair(lo, x[0], x[1]);
        unpair(hi, x[2], x[3]);
    }
};
__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) { return {fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ Vec<4> fma(Vec<4> a, Vec<4> b, Vec<4> c) {
    return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)};
}
__device__ __forceinline__ Vec<1> mul(Vec<1> a, Vec<1> b) { return {__fmul_rn(a.v, b.v)}; }
__device__ __forceinline__ Vec<4> mul(Vec<4> a, Vec<4> b) {
    return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)};
}
// A product that the compiler does not join with the sum that follows, as it may with a
// pair's: it does so in scan_short_bwd_kernel.
__device__ __forceinline__ Vec<1> mul_alone(Vec<1> a, Vec<1> b) { return mul(a, b); }
__device__ __forceinline__ Vec<4> mul_alone(Vec<4> a, Vec<4> b) {
    float x[4], y[4];
    a.to(x);
    b.to(y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __fmul_rn(x[i], y[i]);
    return Vec<4>::of(x);
}
__device__ __forceinline__ Vec<1> add(Vec<1> a, Vec<1> b) { return {__fadd_rn(a.v, b.v)}; }
__device__ __forceinline__ Vec<4> add(Vec<4> a, Vec<4> b) {
    return {add2(a.lo, b.lo), add2(a.hi, b.hi)};
}

template <int VEC>
__device__ __forceinline__ Vec<VEC> fetch_vec(const float *p) {
    float v[VEC];
    fetch<VEC>(p, v);
    return Vec<VEC>::of(v);
}
template <int VEC, typename E>
__device__ __forceinline__ void store_vec(E *p, const Vec<VEC> &x) {
    float v[VEC];
    x.to(v);
    store<VEC>(p, v);
}
template <typename E, int VEC>
__device__ __forceinline__ Vec<VEC> widen(const Raw<E, VEC> &r) {
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r.at(i);
    return Vec<VEC>::of(v);
}

// exp(l), within 2 roundings of 2^-24 and with no lean to either side: a channel of
// long memory multiplies hundreds of gates near 1, where the hardware's 2^x, low by a
// third of a rounding on average, takes fp32 states from 5e-7 to 3e-6 off.
// l = n ln 2 + r by Cody and Waite's two-part reduction (ln 2 = 355/512 + the rest),
// e^r = 1 + r (1 + r q(r)) with q the degree-4 Chebyshev fit of (e^r - 1 - r) / r^2 on
// |r| <= ln 2 / 2 (off by 0.18 roundings at most), and 2^n, which is exact and 0 below
// 2^-126.  Gates below exp(-1000) are 0, -infinity among them; a NaN stays one.
template <int VEC>
__device__ __forceinline__ Vec<VEC> gate(const Raw<float, VEC> &raw) {
    using V = Vec<VEC>;
    float l[VEC], e[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(l[i]) : "f"(raw.at(i)), "f"(-1000.f));
    const V x = V::of(l);
    // adding 3 * 2^22 rounds to a whole number
    const V n = add(fma(x, V::all(1.4426950408889634f), V::all(12582912.f)), V::all(-12582912.f));
    const V r = fma(n, V::all(2.1219444005469057e-4f), fma(n, V::all(-0.693359375f), x));
    V q = fma(V::all(1.3926213141530752e-3f), r, V::all(8.363203145563602e-3f));
    q = fma(q, r, V::all(4.1666556149721146e-2f));
    q = fma(q, r, V::all(0.16666576266288757f));
    q = fma(q, r, V::all(0.5f));
    q = fma(fma(q, r, V::all(1.f)), r, V::all(1.f));
    n.to(e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(e[i]));
    return mul(q, V::of(e));
}

// ---------------------------------------------------------------- exchange in the cluster

// What the blocks of a cluster tell each other of a tile: per channel, the pair
// (P, H) of the map s -> P s + H over the block's whole tile.
//
// A block sends its pairs of tile k with stores that count as bytes of the receiver's
// barrier, so that neither side waits for its other memory traffic.  Two buffers in
// turn are enough.  Who sends tile k has passed a __syncthreads after its block's wait for
// tile k - 1, so every block has sent its pairs of tile k - 1; and it sent them after a
// __syncthreads that follows its own reads of tile k - 2, the last ones of the buffer that
// tile k uses.
constexpr int kBuffers = 2;

template <int CH>
struct Exchange {
    float2 pair[kBuffers][cluster_of(CH)][CH];
    uint64_t bar[kBuffers];
};

template <int CH>
__device__ __forceinline__ void exchange_init(Exchange<CH> &x, unsigned cl) {
    if (cl == 1) return;
    if (threadIdx.x == 0) {
        for (int b = 0; b < kBuffers; ++b) mbar_init(&x.bar[b], 1);
        fence_mbar_init();
    }
    __syncwarp();
    cluster_sync_all();
}

// Sends block `rank`'s pair of channel c for the tile of buffer b to every block.
template <int CH>
__device__ __forceinline__ void exchange_send(Exchange<CH> &x, int b, unsigned rank, unsigned cl,
                                              int c, float P, float H) {
    if (c == 0) mbar_arrive_expect_tx(&x.bar[b], cl * CH * sizeof(float2));
    const uint32_t at = smem_u32(&x.pair[b][rank][c]), bar = smem_u32(&x.bar[b]);
    for (unsigned j = 0; j < cl; ++j)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                         mapa_shared(at, j)),
                     "f"(P), "f"(H), "r"(mapa_shared(bar, j))
                     : "memory");
}

__device__ __forceinline__ bool exchange_done(uint64_t *bar, unsigned parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// Waits for every block's pairs of buffer b, the n-th tile that uses it.  After a wait that
// ran out (`*dead`) no other is made: the status word says so, the results are
// unspecified, and every block still comes to its end.
template <int CH>
__device__ __forceinline__ void exchange_wait(Exchange<CH> &x, int b, unsigned n, bool *dead,
                                              unsigned *status) {
    if (*dead || exchange_done(&x.bar[b], n & 1)) return;
    const unsigned long long start = global_timer_ns();
    while (!exchange_done(&x.bar[b], n & 1)) {
        if (global_timer_ns() - start > kWaitLimitNs) {
            atomicOr(status, kStatusTimeout);
            *dead = true;
            return;
        }
    }
}

// No block leaves while another may still send to it.
__device__ __forceinline__ void exchange_end(unsigned cl) {
    if (cl > 1)
        asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// ---------------------------------------------------------------- tiles on their way

// Waits for the phase with this parity of a barrier that bulk copies complete.  After a wait
// that ran out (`*dead`) no other is made.
__device__ __forceinline__ void copy_wait(uint64_t *bar, unsigned parity, bool *dead,
                                          unsigned *status) {
    if (!*dead && !mbar_wait_bounded(bar, parity & 1, status)) *dead = true;
}

// After a wait that ran out: one more bounded wait for the last copies into each stage, so that
// none is in flight when the block ends.
template <int STAGES>
__device__ __forceinline__ void copies_drain(uint64_t *bars, unsigned tiles, unsigned *status) {
    for (int i = 0; i < STAGES; ++i)
        if (tiles > static_cast<unsigned>(i))
            mbar_wait_bounded(&bars[i], ((tiles - 1 - i) / (STAGES ? STAGES : 1)) & 1, status);
}

// One stage of the forward's queue: a tile of log_alpha and x as TMA lays it down.  Rows and
// channels outside the tensor arrive as zeros, a gate of 1 and an x of 0, which change nothing.
template <typename E, int CH, int TOKENS>
struct FwdStage {
    float l[TOKENS][CH];
    E x[TOKENS][CH];
    static constexpr unsigned kBytes = TOKENS * CH * (4 + sizeof(E));
};
template <typename E, int CH, int TOKENS>
struct BwdStage {
    float l[TOKENS][CH];
    E x[TOKENS][CH], d[TOKENS][CH];
    static constexpr unsigned kBytes = TOKENS * CH * (4 + 2 * sizeof(E));
};

template <typename V>
__device__ __forceinline__ void keep_if(bool there, V &x, const V &otherwise) {
    if (!there) x = otherwise;
}

// A thread's tokens of one tile, in registers.
template <typename E, int VEC, int TPW>
struct FwdTokens {
    Vec<VEC> a[TPW], x[TPW];
};
template <typename E, int VEC, int TPW>
struct BwdTokens {
    Vec<VEC> a[TPW];
    Raw<E, VEC> x[TPW], d[TPW];
};

// Forward.  Per tile: each run reduces its tokens to the pair (P, H) that maps
// the state before them to the state after them, h -> P h + H; the runs' pairs
// are scanned in the block, the blocks' pairs exchanged in the cluster, and each
// run walks its tokens again from its true state, from registers.
//
// Two things run ahead of the walk.  The next STAGES tiles are on their way to shared
// memory (STAGES = 0: the next one to registers).  And tile k is reduced before tile k - 1
// is walked, so that the exchange has a whole tile's time and one barrier a tile is enough
// (B1 T262144 D1024 by cluster barriers, which wait for a block's stores too: 542 us).
template <typename E, int VEC, int LPR, int TPW, int THREADS, int STAGES>
__global__ void __launch_bounds__(THREADS, 2)
    scan_fwd_kernel(const __grid_constant__ ScanArgs p) {
    using G = Tile<VEC, LPR, TPW, THREADS>;
    using Set = FwdTokens<E, VEC, TPW>;
    using V = Vec<VEC>;
    constexpr int CH = G::kChannels, RUNS = G::kRuns;
    using Stage = FwdStage<E, CH, G::kTokens>;
    extern __shared__ __align__(128) unsigned char s_dynamic[];
    Stage *stages = reinterpret_cast<Stage *>(s_dynamic);
    __shared__ __align__(16) float s_p[2][RUNS][CH], s_h[2][RUNS][CH];
    __shared__ __align__(16) float s_start[2][CH];   // the states that enter the block's tiles
    __shared__ __align__(16) Exchange<CH> s_x;
    __shared__ __align__(8) uint64_t s_full[STAGES ? STAGES : 1];
    const int tid = threadIdx.x, run = tid / LPR, cl0 = (tid % LPR) * VEC;
    const Place o = place<G, VEC, LPR>(p);
    if (o.len == 0) {
        if (p.hT && o.valid && o.rank == 0 && run == 0)
            store_vec<VEC>(p.hT + o.state, p.h0 ? fetch_vec<VEC>(p.h0 + o.state) : V::all(0.f));
        return;
    }
    const unsigned span = o.cl * G::kTokens;
    const unsigned mine = o.rank * G::kTokens + run * TPW;   // this thread's tokens of a tile
    const unsigned tiles = (o.len - 1) / span + 1;
    // The last CH threads scan a channel each over the block's runs.  They, or in a
    // cluster the first CH, carry its state from tile to tile.
    const int sc = tid % CH;
    float carry = 0.f;
    if (p.h0 && o.first + sc < p.D) carry = p.h0[o.state - cl0 + sc];
    bool dead = false;

    // one thread asks for tile k; a block whose part of it is past the end only ends the phase
    const auto asked = [&](unsigned k) { return k * span + o.rank * G::kTokens < o.len; };
    const auto request = [&](unsigned k, int stage) {
        if (STAGES == 0 || tid != 0 || k >= tiles) return;
        if (!asked(k)) {
            mbar_arrive(&s_full[stage]);
        } else {
            const int row = static_cast<int>(o.start + k * span + o.rank * G::kTokens);
            mbar_arrive_expect_tx(&s_full[stage], Stage::kBytes);
            tma_load_3d(&stages[stage].l[0][0], &p.map_l, &s_full[stage], o.first, row, o.head);
            tma_load_3d(&stages[stage].x[0][0], &p.map_x, &s_full[stage], o.first, row, o.head);
        }
    };
    if constexpr (STAGES > 0) {
        if (tid == 0) {
            for (int i = 0; i < STAGES; ++i) mbar_init(&s_full[i], 1);
            fence_mbar_init();
            for (int i = 0; i < STAGES; ++i) request(i, i);
        }
    }
    exchange_init<CH>(s_x, o.cl);
    __syncthreads();

    // without TMA: the next tile's values on their way to registers
    Raw<float, VEC> l_next[TPW];
    Raw<E, VEC> x_next[TPW];
    const auto ahead = [&](unsigned k) {
        const unsigned t0 = k * span + mine;
        const size_t at = o.row + static_cast<size_t>(t0) * p.D;
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
            x_next[i] = Raw<E, VEC>{};
            l_next[i] = Raw<float, VEC>{};
            if (o.valid && k < tiles && t0 + i < o.len) {
                l_next[i] = load<float, VEC>(p.log_alpha, at + static_cast<size_t>(i) * p.D);
                x_next[i] = load<E, VEC>(p.x, at + static_cast<size_t>(i) * p.D);
            }
        }
    };
    if constexpr (STAGES == 0) ahead(0);

    int stage = 0;
    unsigned turn = 0;   // parity of the stage's phase
    const auto reduce = [&](unsigned k, Set &c, float (*sp)[CH], float (*sh)[CH]) {
        const unsigned t0 = k * span + mine;
        if constexpr (STAGES > 0) {
            const Stage &st = stages[stage];
            if (asked(k)) {
                copy_wait(&s_full[stage], turn, &dead, p.status);
#pragma unroll
                for (int i = 0; i < TPW; ++i) {
                    c.a[i] = gate<VEC>(load<float, VEC>(&st.l[run * TPW + i][cl0], 0));
                    c.x[i] = widen(load<E, VEC>(&st.x[run * TPW + i][cl0], 0));
                }
                if (t0 + TPW > o.len) {   // the rows of the next sequence, if any
#pragma unroll
                    for (int i = 0; i < TPW; ++i) {
                        keep_if(t0 + i < o.len, c.a[i], V::all(1.f));
                        keep_if(t0 + i < o.len, c.x[i], V::all(0.f));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < TPW; ++i) c.a[i] = V::all(1.f), c.x[i] = V::all(0.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < TPW; ++i) c.a[i] = gate<VEC>(l_next[i]), c.x[i] = widen(x_next[i]);
            ahead(k + 1);
        }
        V P = c.a[0], H = c.x[0];
#pragma unroll
        for (int i = 1; i < TPW; ++i) {
            H = fma(c.a[i], H, c.x[i]);
            P = mul(P, c.a[i]);
        }
        store_vec<VEC>(&sp[run][cl0], P);
        store_vec<VEC>(&sh[run][cl0], H);
    };
    // the state that enters this block's part of tile k, and on to the next tile
    const auto enter = [&](unsigned k, float *start_of) {
        if (tid >= CH) return;
        const int b = k % kBuffers;
        exchange_wait<CH>(s_x, b, k / kBuffers, &dead, p.status);
        float start = carry;
        for (unsigned j = 0; j < o.cl; ++j) {
            const float2 q = s_x.pair[b][j][tid];
            if (j == o.rank) start = carry;
            carry = fmaf(q.x, carry, q.y);
        }
        start_of[tid] = start;
    };
    // the block's own scan over its runs of tile k
    const auto scan = [&](unsigned k, float (*sp)[CH], float (*sh)[CH], float *start_of) {
        if (tid < THREADS - CH) return;
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
            const float rp = sp[r][sc], rh = sh[r][sc];
            sp[r][sc] = P;
            sh[r][sc] = H;
            H = fmaf(rp, H, rh);
            P *= rp;
        }
        if (o.cl == 1) {
            start_of[sc] = carry;
            carry = fmaf(P, carry, H);
        } else {
            exchange_send<CH>(s_x, k % kBuffers, o.rank, o.cl, sc, P, H);
        }
    };
    const size_t pitch = p.D;
    const auto walk = [&](unsigned k, const Set &c, float (*sp)[CH], float (*sh)[CH],
                          const float *start_of) {
        const unsigned t0 = k * span + mine;
        if (!o.valid || t0 >= o.len) return;
        V h = fma(fetch_vec<VEC>(&sp[run][cl0]), fetch_vec<VEC>(&start_of[cl0]),
                  fetch_vec<VEC>(&sh[run][cl0]));
        if (p.ckpt_out && t0 % kBlock == 0)
            store_vec<VEC>(p.ckpt_out + o.ck + (t0 / kBlock) * pitch, h);
        E *out = static_cast<E *>(p.h) + (o.row + t0 * pitch);
        if (p.h && t0 + TPW <= o.len) {
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
                h = fma(c.a[i], h, c.x[i]);
                store_vec<VEC>(out, h);
                out += pitch;
            }
        } else {
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
                h = fma(c.a[i], h, c.x[i]);
                if (p.h && t0 + i < o.len) store_vec<VEC>(out, h);
                out += pitch;
            }
        }
        if (p.hT && o.len - t0 <= TPW) store_vec<VEC>(p.hT + o.state, h);
    };

    const auto step = [&](unsigned k, Set &now, const Set &last, auto parity) {
        constexpr int B = decltype(parity)::value;
        reduce(k, now, s_p[B], s_h[B]);
        if (o.cl > 1 && k > 0) enter(k - 1, s_start[B ^ 1]);
        __syncthreads();
        request(k + STAGES, stage);   // every thread has read its part of the stage
        if (++stage == STAGES) stage = 0, ++turn;
        scan(k, s_p[B], s_h[B], s_start[B]);
        if (k > 0) walk(k - 1, last, s_p[B ^ 1], s_h[B ^ 1], s_start[B ^ 1]);
    };
    Set even, odd;
    unsigned k = 0;
    for (; k + 1 < tiles; k += 2) {
        step(k, even, odd, std::integral_constant<int, 0>{});
        step(k + 1, odd, even, std::integral_constant<int, 1>{});
    }
    if (k < tiles) step(k, even, odd, std::integral_constant<int, 0>{});
    const int B = (tiles - 1) & 1;
    if (o.cl > 1) enter(tiles - 1, s_start[B]);
    __syncthreads();
    if (B == 0) walk(tiles - 1, even, s_p[0], s_h[0], s_start[0]);
    else walk(tiles - 1, odd, s_p[1], s_h[1], s_start[1]);
    if (STAGES > 0 && dead && tid == 0) copies_drain<STAGES>(s_full, tiles, p.status);
    exchange_end(o.cl);
}

// Backward, from the last tile to the first, in the same way: tile k counts from the end.
// Forward in time, the states h_{t-1} are walked again from the checkpoint of each
// block of kBlock tokens; backward in time, u_t = alpha_t g_t is the recurrence's
// own scan from the end: a run maps the u that enters it on the right to the one that
// leaves it on the left, u -> P u + U, with the same P.  The walk's products (mul_alone) and
// sums are rounded one by one in both of its loops, so that a call with fewer outputs gives
// the same bits.
template <typename E, int VEC, int LPR, int TPW, int THREADS, int STAGES>
__global__ void __launch_bounds__(THREADS, STAGES == 0 && VEC == 4 ? 1 : 2)
    scan_bwd_kernel(const __grid_constant__ ScanArgs p) {
    using G = Tile<VEC, LPR, TPW, THREADS>;
    using Set = BwdTokens<E, VEC, TPW>;
    using V = Vec<VEC>;
    constexpr int CH = G::kChannels, RUNS = G::kRuns;
    constexpr int RPB = kBlock / TPW, BLOCKS = RUNS / RPB;   // runs of a block, blocks of a tile
    static_assert(RUNS % RPB == 0 && 3 * CH <= THREADS, "whole blocks, three scans side by side");
    using Stage = BwdStage<E, CH, G::kTokens>;
    extern __shared__ __align__(128) unsigned char s_dynamic[];
    Stage *stages = reinterpret_cast<Stage *>(s_dynamic);
    __shared__ __align__(16) float s_p[2][RUNS][CH], s_start[2][CH];
    __shared__ __align__(16) float s_h[2][RUNS][CH];   // a run's H, then the state that enters it
    __shared__ __align__(16) float s_u[2][RUNS][CH];   // a run's U, then that of the runs to its right
    __shared__ __align__(16) float s_q[2][RUNS][CH];   // the P of the runs to its right
    __shared__ __align__(16) Exchange<CH> s_x;
    __shared__ __align__(8) uint64_t s_full[STAGES ? STAGES : 1];
    const int tid = threadIdx.x, run = tid / LPR, cl0 = (tid % LPR) * VEC;
    const Place o = place<G, VEC, LPR>(p);
    if (o.len == 0) {
        if (p.hT && o.valid && o.rank == 0 && run == 0)
            store_vec<VEC>(p.hT + o.state, p.dhT ? fetch_vec<VEC>(p.dhT + o.state) : V::all(0.f));
        return;
    }
    const unsigned span = o.cl * G::kTokens;
    const unsigned mine = o.rank * G::kTokens + run * TPW;
    const unsigned tiles = (o.len - 1) / span + 1;
    // one channel to a thread: the last CH scan u over the block's runs, the CH before them
    // h; the last, or in a cluster the first CH, carry u from tile to tile
    const int sc = tid % CH;
    const bool there_c = o.first + sc < p.D;
    const bool scan_h = tid >= THREADS - 2 * CH && tid < THREADS - CH;
    const float *ck = p.ckpt_in + (o.ck - cl0 + sc);
    float carry = 0.f;
    if (p.dhT && there_c) carry = p.dhT[o.state - cl0 + sc];
    bool dead = false;

    const auto base_of = [&](unsigned k) { return (tiles - 1 - k) * span; };
    const auto asked = [&](unsigned k) { return base_of(k) + o.rank * G::kTokens < o.len; };
    const auto request = [&](unsigned k, int stage) {
        if (STAGES == 0 || tid != 0 || k >= tiles) return;
        if (!asked(k)) {
            mbar_arrive(&s_full[stage]);
        } else {
            const int row = static_cast<int>(o.start + base_of(k) + o.rank * G::kTokens);
            mbar_arrive_expect_tx(&s_full[stage],
                                  Stage::kBytes - (p.d_h ? 0 : sizeof(stages[0].d)));
            tma_load_3d(&stages[stage].l[0][0], &p.map_l, &s_full[stage], o.first, row, o.head);
            tma_load_3d(&stages[stage].x[0][0], &p.map_x, &s_full[stage], o.first, row, o.head);
            if (p.d_h)
                tma_load_3d(&stages[stage].d[0][0], &p.map_d, &s_full[stage], o.first, row, o.head);
        }
    };
    if constexpr (STAGES > 0) {
        if (tid == 0) {
            for (int i = 0; i < STAGES; ++i) mbar_init(&s_full[i], 1);
            fence_mbar_init();
            for (int i = 0; i < STAGES; ++i) request(i, i);
        }
    }
    exchange_init<CH>(s_x, o.cl);
    __syncthreads();

    // the checkpoints of tile k for the threads that scan h, one tile ahead
    const auto checkpoints = [&](unsigned k, float (&e)[BLOCKS]) {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const unsigned t = base_of(k) + o.rank * G::kTokens + b * kBlock;
            e[b] = scan_h && there_c && k < tiles && t < o.len
                       ? ck[static_cast<size_t>(t / kBlock) * p.D] : 0.f;
        }
    };
    float enters[BLOCKS], next[BLOCKS];
    checkpoints(0, next);

    // without TMA: the next tile's values on their way to registers
    Raw<float, VEC> l_next[TPW];
    Raw<E, VEC> x_next[TPW], d_next[TPW];
    const auto ahead = [&](unsigned k) {
        const unsigned t0 = base_of(k) + mine;
        const size_t at = o.row + static_cast<size_t>(t0) * p.D;
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
            x_next[i] = d_next[i] = Raw<E, VEC>{};
            l_next[i] = Raw<float, VEC>{};
            if (o.valid && k < tiles && t0 + i < o.len) {
                const size_t e = at + static_cast<size_t>(i) * p.D;
                l_next[i] = load<float, VEC>(p.log_alpha, e);
                x_next[i] = load<E, VEC>(p.x, e);
                if (p.d_h) d_next[i] = load<E, VEC>(p.d_h, e);
            }
        }
    };
    if constexpr (STAGES == 0) ahead(0);

    int stage = 0;
    unsigned turn = 0;   // parity of the stage's phase
    const auto reduce = [&](unsigned k, Set &c, float (*sp)[CH], float (*sh)[CH],
                            float (*su)[CH]) {
        const unsigned t0 = base_of(k) + mine;
#pragma unroll
        for (int i = 0; i < TPW; ++i) c.d[i] = Raw<E, VEC>{};
        if constexpr (STAGES > 0) {
            const Stage &st = stages[stage];
            if (asked(k)) {
                copy_wait(&s_full[stage], turn, &dead, p.status);
#pragma unroll
                for (int i = 0; i < TPW; ++i) {
                    c.a[i] = gate<VEC>(load<float, VEC>(&st.l[run * TPW + i][cl0], 0));
                    c.x[i] = load<E, VEC>(&st.x[run * TPW + i][cl0], 0);
                }
                if (p.d_h) {
#pragma unroll
                    for (int i = 0; i < TPW; ++i) c.d[i] = load<E, VEC>(&st.d[run * TPW + i][cl0], 0);
                }
                if (t0 + TPW > o.len) {   // the rows of the next sequence, if any
#pragma unroll
                    for (int i = 0; i < TPW; ++i) {
                        keep_if(t0 + i < o.len, c.a[i], V::all(1.f));
                        keep_if(t0 + i < o.len, c.x[i], Raw<E, VEC>{});
                        keep_if(t0 + i < o.len, c.d[i], Raw<E, VEC>{});
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < TPW; ++i) c.a[i] = V::all(1.f), c.x[i] = Raw<E, VEC>{};
            }
        } else {
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
                c.a[i] = gate<VEC>(l_next[i]);
                c.x[i] = x_next[i];
                c.d[i] = d_next[i];
            }
            ahead(k + 1);
        }
        V P = c.a[0], H = widen(c.x[0]), U = mul(c.a[TPW - 1], widen(c.d[TPW - 1]));
#pragma unroll
        for (int i = 1; i < TPW; ++i) {
            H = fma(c.a[i], H, widen(c.x[i]));
            P = mul(P, c.a[i]);
            U = mul(c.a[TPW - 1 - i], add(U, widen(c.d[TPW - 1 - i])));
        }
        store_vec<VEC>(&sp[run][cl0], P);
        store_vec<VEC>(&sh[run][cl0], H);
        store_vec<VEC>(&su[run][cl0], U);
    };
    // the u that enters this block's part of tile k from the right, and on to the next tile
    const auto enter = [&](unsigned k, float *start_of) {
        if (tid >= CH) return;
        const int b = k % kBuffers;
        exchange_wait<CH>(s_x, b, k / kBuffers, &dead, p.status);
        float start = carry;
        for (unsigned j = o.cl; j-- > 0;) {
            const float2 q = s_x.pair[b][j][tid];
            if (j == o.rank) start = carry;
            carry = fmaf(q.x, carry, q.y);
        }
        start_of[tid] = start;
    };
    const auto scan = [&](unsigned k, float (*sp)[CH], float (*sh)[CH], float (*su)[CH],
                          float (*sq)[CH], float *start_of) {
        if (scan_h) {
            float h = 0.f;
#pragma unroll 8
            for (int r = 0; r < RUNS; ++r) {
                if (r % RPB == 0) h = enters[r / RPB];
                const float H = sh[r][sc];
                sh[r][sc] = h;
                h = fmaf(sp[r][sc], h, H);
            }
        } else if (tid >= THREADS - CH) {
            float P = 1.f, U = 0.f;
#pragma unroll 8
            for (int r = RUNS - 1; r >= 0; --r) {
                const float rp = sp[r][sc], ru = su[r][sc];
                su[r][sc] = U;
                sq[r][sc] = P;
                U = fmaf(rp, U, ru);
                P *= rp;
            }
            if (o.cl == 1) {
                start_of[sc] = carry;
                carry = fmaf(P, carry, U);
            } else {
                exchange_send<CH>(s_x, k % kBuffers, o.rank, o.cl, sc, P, U);
            }
        }
    };
    const size_t pitch = p.D;
    const auto walk = [&](unsigned k, const Set &c, float (*sh)[CH], float (*su)[CH],
                          float (*sq)[CH], const float *start_of) {
        const unsigned t0 = base_of(k) + mine;
        if (!o.valid || t0 >= o.len) return;
        V u = fma(fetch_vec<VEC>(&sq[run][cl0]), fetch_vec<VEC>(&start_of[cl0]),
                  fetch_vec<VEC>(&su[run][cl0]));
        V before[TPW];
        before[0] = fetch_vec<VEC>(&sh[run][cl0]);
#pragma unroll
        for (int i = 1; i < TPW; ++i) before[i] = fma(c.a[i - 1], before[i - 1], widen(c.x[i - 1]));
        const size_t last = o.row + (t0 + TPW - 1) * pitch;
        E *dx = static_cast<E *>(p.h) + last;
        float *da = p.ga + last;
        if (p.h && p.ga && t0 + TPW <= o.len) {
#pragma unroll
            for (int i = TPW - 1; i >= 0; --i) {
                const V g = add(u, widen(c.d[i]));
                u = mul_alone(c.a[i], g);
                store_vec<VEC>(dx, g);
                store_vec<VEC>(da, mul(u, before[i]));
                dx -= pitch;
                da -= pitch;
            }
        } else {
#pragma unroll
            for (int i = TPW - 1; i >= 0; --i) {
                const V g = add(u, widen(c.d[i]));
                u = mul_alone(c.a[i], g);
                if (p.h && t0 + i < o.len) store_vec<VEC>(dx, g);
                if (p.ga && t0 + i < o.len) store_vec<VEC>(da, mul(u, before[i]));
                dx -= pitch;
                da -= pitch;
            }
        }
        if (p.hT && t0 == 0) store_vec<VEC>(p.hT + o.state, u);
    };

    const auto step = [&](unsigned k, Set &now, const Set &last, auto parity) {
        constexpr int B = decltype(parity)::value;
        reduce(k, now, s_p[B], s_h[B], s_u[B]);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) enters[b] = next[b];
        checkpoints(k + 1, next);
        if (o.cl > 1 && k > 0) enter(k - 1, s_start[B ^ 1]);
        __syncthreads();
        request(k + STAGES, stage);   // every thread has read its part of the stage
        if (++stage == STAGES) stage = 0, ++turn;
        scan(k, s_p[B], s_h[B], s_u[B], s_q[B], s_start[B]);
        if (k > 0) walk(k - 1, last, s_h[B ^ 1], s_u[B ^ 1], s_q[B ^ 1], s_start[B ^ 1]);
    };
    Set even, odd;
    unsigned k = 0;
    for (; k + 1 < tiles; k += 2) {
        step(k, even, odd, std::integral_constant<int, 0>{});
        step(k + 1, odd, even, std::integral_constant<int, 1>{});
    }
    if (k < tiles) step(k, even, odd, std::integral_constant<int, 0>{});
    const int B = (tiles - 1) & 1;
    if (o.cl > 1) enter(tiles - 1, s_start[B]);
    __syncthreads();
    if (B == 0) walk(tiles - 1, even, s_h[0], s_u[0], s_q[0], s_start[0]);
    else walk(tiles - 1, odd, s_h[1], s_u[1], s_q[1], s_start[1]);
    if (STAGES > 0 && dead && tid == 0) copies_drain<STAGES>(s_full, tiles, p.status);
    exchange_end(o.cl);
}

// Short sequences: a thread walks one by itself, VEC channels of it, kChunk tokens on their
// way at a time.  No tile to fill, no exchange.
constexpr int kShortThreads = 64;

struct ShortPlace {
    int len;
    size_t row, state, ck;   // elements: first row, state and checkpoint of its channels
};

template <int VEC>
__device__ __forceinline__ bool short_place(const ScanArgs &p, ShortPlace &o) {
    const unsigned i = blockIdx.x * kShortThreads + threadIdx.x;
    const unsigned pieces = p.D / VEC, unit = i / pieces, c = (i % pieces) * VEC;
    if (unit >= static_cast<unsigned>(p.nseq) * p.H) return false;
    const unsigned head = unit % p.H;
    const ScanSeq s = p.seqs[unit / p.H];
    o.len = s.len;
    o.row = (static_cast<size_t>(head) * p.rows + s.first) * p.D + c;
    o.state = (static_cast<size_t>(s.n) * p.H + head) * p.D + c;
    o.ck = (static_cast<size_t>(head) * p.blocks + s.block) * p.D + c;
    return true;
}

template <typename E, int VEC>
struct ShortChunk {
    Raw<float, VEC> l[kChunk];
    Raw<E, VEC> x[kChunk];
    __device__ __forceinline__ void read(const ScanArgs &p, const ShortPlace &o, int t0) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            l[i] = Raw<float, VEC>{};
            x[i] = Raw<E, VEC>{};
            if (t0 + i >= o.len) continue;
            const size_t at = o.row + static_cast<size_t>(t0 + i) * p.D;
            l[i] = load<float, VEC>(p.log_alpha, at);
            x[i] = load<E, VEC>(p.x, at);
        }
    }
};

template <typename E, int VEC>
__global__ void __launch_bounds__(kShortThreads)
    scan_short_fwd_kernel(const __grid_constant__ ScanArgs p) {
    using V = Vec<VEC>;
    ShortPlace o;
    if (!short_place<VEC>(p, o)) return;
    ShortChunk<E, VEC> c;
    c.read(p, o, 0);
    V h = p.h0 ? fetch_vec<VEC>(p.h0 + o.state) : V::all(0.f);
    for (int t0 = 0; t0 < o.len; t0 += kChunk) {
        if (p.ckpt_out && t0 % kBlock == 0)
            store_vec<VEC>(p.ckpt_out + o.ck + static_cast<size_t>(t0 / kBlock) * p.D, h);
        V a[kChunk], x[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) a[i] = gate<VEC>(c.l[i]), x[i] = widen(c.x[i]);
        c.read(p, o, t0 + kChunk);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            h = fma(a[i], h, x[i]);
            if (p.h && t0 + i < o.len)
                store_vec<VEC>(static_cast<E *>(p.h) + (o.row + static_cast<size_t>(t0 + i) * p.D), h);
        }
    }
    if (p.hT) store_vec<VEC>(p.hT + o.state, h);
}

// Backward, a block of the checkpoints after another from the end: the states that enter its
// chunks first, then the chunks from the last.
template <typename E, int VEC>
__global__ void __launch_bounds__(kShortThreads)
    scan_short_bwd_kernel(const __grid_constant__ ScanArgs p) {
    using V = Vec<VEC>;
    ShortPlace o;
    if (!short_place<VEC>(p, o)) return;
    V u = p.dhT ? fetch_vec<VEC>(p.dhT + o.state) : V::all(0.f);
    for (int base = (o.len - 1) / kBlock * kBlock; base >= 0 && o.len > 0; base -= kBlock) {
        const int chunks = (min(o.len - base, kBlock) + kChunk - 1) / kChunk;
        ShortChunk<E, VEC> c;
        Raw<E, VEC> d[kChunk];
        const auto read_d = [&](int t0) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                d[i] = Raw<E, VEC>{};
                if (p.d_h && t0 + i < o.len)
                    d[i] = load<E, VEC>(p.d_h, o.row + static_cast<size_t>(t0 + i) * p.D);
            }
        };
        c.read(p, o, base);
        V state[kBlock / kChunk];
        state[0] = fetch_vec<VEC>(p.ckpt_in + o.ck + static_cast<size_t>(base / kBlock) * p.D);
        for (int k = 0; k + 1 < chunks; ++k) {
            V a[kChunk], x[kChunk];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) a[i] = gate<VEC>(c.l[i]), x[i] = widen(c.x[i]);
            c.read(p, o, base + (k + 1) * kChunk);
            V h = state[k];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) h = fma(a[i], h, x[i]);
            state[k + 1] = h;
        }
        read_d(base + (chunks - 1) * kChunk);
        for (int k = chunks - 1; k >= 0; --k) {
            const int t0 = base + k * kChunk;
            V a[kChunk], before[kChunk], dd[kChunk];
            V h = state[k];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                a[i] = gate<VEC>(c.l[i]);
                before[i] = h;
                h = fma(a[i], h, widen(c.x[i]));
                dd[i] = widen(d[i]);
            }
            if (k > 0) {
                c.read(p, o, t0 - kChunk);
                read_d(t0 - kChunk);
            }
#pragma unroll
            for (int i = kChunk - 1; i >= 0; --i) {
                const V g = add(u, dd[i]);
                u = mul_alone(a[i], g);
                if (t0 + i >= o.len) continue;
                const size_t at = o.row + static_cast<size_t>(t0 + i) * p.D;
                if (p.h) store_vec<VEC>(static_cast<E *>(p.h) + at, g);
                if (p.ga) store_vec<VEC>(p.ga + at, mul(u, before[i]));
            }
        }
    }
    if (p.hT) store_vec<VEC>(p.hT + o.state, u);
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

// Whether two tensors of n elements each share memory without being the same elements: a
// thread that reads and writes its own element of both would then meet another thread's.
bool mixed(const void *a, int size_a, const void *b, int size_b, long long n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(n) * size_b && y < x + static_cast<uintptr_t>(n) * size_a &&
           (x != y || size_a != size_b);
}

// Checks shared by the scans; cu_seqlens [N + 1] is checked by the caller's loop.
int check_common(const ScanArgs &a, long long states, int D, int dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_ARG;
    if (!elements_aligned(a, dtype)) return GLA_ERR_ARG;
    // thread blocks of the narrowest tiles in the longest clusters
    if (states > 0x7fffffffLL / kMaxCluster / ((D + 31LL) / 32)) return GLA_ERR_ARG;
    return GLA_OK;
}

// Launches Kernel over the units of `a` in clusters of a.cluster thread blocks.
template <typename G, auto Kernel>
int launch(const ScanArgs &a, size_t dynamic, cudaStream_t stream) {
    const long long units =
        static_cast<long long>(a.nseq) * a.H * ((a.D + G::kChannels - 1) / G::kChannels);
    // once for each device
    static std::atomic<unsigned long long> allowed{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return static_cast<int>(cudaGetLastError());
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(dynamic));
        if (e == cudaSuccess)   // clusters of more than 8
            e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return static_cast<int>(e);
        allowed.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(a.cluster), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * a.cluster));
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = dynamic;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, Kernel, a));
}

template <typename E, int VEC, int LPR, int TPW, int THREADS, int STAGES>
int launch_fwd(const ScanArgs &a, cudaStream_t stream) {
    using G = Tile<VEC, LPR, TPW, THREADS>;
    return launch<G, scan_fwd_kernel<E, VEC, LPR, TPW, THREADS, STAGES>>(
        a, STAGES * sizeof(FwdStage<E, G::kChannels, G::kTokens>), stream);
}

template <typename E, int VEC, int LPR, int TPW, int THREADS, int STAGES>
int launch_bwd(const ScanArgs &a, cudaStream_t stream) {
    using G = Tile<VEC, LPR, TPW, THREADS>;
    return launch<G, scan_bwd_kernel<E, VEC, LPR, TPW, THREADS, STAGES>>(
        a, STAGES * sizeof(BwdStage<E, G::kChannels, G::kTokens>), stream);
}

template <typename E>
int launch_for(ScanArgs &a, bool backward, Way way, cudaStream_t stream) {
    if (way == Way::kOne) return backward ? launch_bwd<E, 1, 32, 8, 256, 0>(a, stream)
                                          : launch_fwd<E, 1, 32, 8, 256, 0>(a, stream);
    if constexpr (sizeof(E) == 2)   // four fp32 values are a piece that TMA takes
        if (way == Way::kFour) return backward ? launch_bwd<E, 4, 8, 4, 256, 0>(a, stream)
                                               : launch_fwd<E, 4, 8, 4, 256, 0>(a, stream);
    const int tokens = 4096 / a.width;
    const bool f32 = sizeof(E) == 4;
    const long long dims[3] = {a.D, a.rows, a.H};
    if (!tile_map(&a.map_l, a.log_alpha, true, dims, a.width, tokens) ||
        !tile_map(&a.map_x, a.x, f32, dims, a.width, tokens) ||
        (a.d_h && !tile_map(&a.map_d, a.d_h, f32, dims, a.width, tokens)))
        return static_cast<int>(cudaErrorInvalidValue);
    if (backward) return launch_bwd<E, 4, 8, 8, 128, 2>(a, stream);
    if (a.width == 128) return launch_fwd<E, 4, 32, 4, 256, 3>(a, stream);
    if (a.width == 64) return launch_fwd<E, 4, 16, 4, 256, 3>(a, stream);
    return launch_fwd<E, 4, 8, 8, 128, 2>(a, stream);
}

template <typename E>
int launch_short(const ScanArgs &a, bool backward, bool vec4, cudaStream_t stream) {
    const long long threads = static_cast<long long>(a.nseq) * a.H * (vec4 ? a.D / 4 : a.D);
    const unsigned grid = static_cast<unsigned>((threads + kShortThreads - 1) / kShortThreads);
    const auto go = [&](auto kernel) {
        kernel<<<grid, kShortThreads, 0, stream>>>(a);
        return static_cast<int>(cudaGetLastError());
    };
    if (backward) return vec4 ? go(scan_short_bwd_kernel<E, 4>) : go(scan_short_bwd_kernel<E, 1>);
    return vec4 ? go(scan_short_fwd_kernel<E, 4>) : go(scan_short_fwd_kernel<E, 1>);
}

// Forward or backward over N sequences of H heads (a fixed-length batch is one
// sequence of B heads).
int run(ScanArgs &a, bool backward, const int *cu_seqlens, int N, int H, int T_total, int D,
        int dtype, cudaStream_t stream) {
    if (!cu_seqlens || N <= 0 || H <= 0 || T_total < 0 || D <= 0) return GLA_ERR_ARG;
    int st = check_common(a, static_cast<long long>(N) * H, D, dtype);
    if (st != GLA_OK) return st;
    if (cu_seqlens[0] != 0 || cu_seqlens[N] != T_total) return GLA_ERR_ARG;
    std::vector<ScanSeq> seqs;
    try {
        seqs.resize(N);
    } catch (const std::bad_alloc &) {   // no exception crosses the C interface
        return GLA_ERR_ALLOC;
    }
    long long blocks = 0;
    for (int n = 0; n < N; ++n) {
        const long long len = static_cast<long long>(cu_seqlens[n + 1]) - cu_seqlens[n];
        if (len < 0) return GLA_ERR_ARG;
        seqs[n] = ScanSeq{cu_seqlens[n], static_cast<int>(len), n, static_cast<int>(blocks)};
        blocks += (len + kBlock - 1) / kBlock;
    }
    int sms = 0;
    st = usable_device(&sms, &a.status);
    if (st != GLA_OK) return st;
    a.rows = T_total;
    a.blocks = blocks;
    a.D = D;
    a.H = H;
    const bool vec4 = D % 4 == 0 && aligned(16, a.x, a.log_alpha, a.h0, a.dhT, a.ckpt_in, a.d_h, a.h,
                                            a.hT, a.ga, a.ckpt_out);
    // TMA wants rows of whole 16-byte pieces
    const Way way = !vec4 ? Way::kOne : dtype == GLA_F32 || D % 8 == 0 ? Way::kTma : Way::kFour;
    // longest first, so that the last thread blocks to start are short ones
    std::stable_sort(seqs.begin(), seqs.end(),
                     [](const ScanSeq &x, const ScanSeq &y) { return x.len > y.len; });
    for (int n = 0; n < N; n += kMaxSeqs) {
        a.nseq = std::min(kMaxSeqs, N - n);
        std::copy(seqs.begin() + n, seqs.begin() + n + a.nseq, a.seqs);
        long long total = 0;
        for (int i = 0; i < a.nseq; ++i) total += a.seqs[i].len;
        const Work work = {static_cast<double>(seqs[n].len), static_cast<double>(total),
                           static_cast<double>(a.nseq), static_cast<double>(H), D,
                           dtype == GLA_BF16 ? 2 : 4, backward, way};
        const Layout plan = layout(work, sms);
        a.width = plan.tiles.width;
        a.cluster = plan.tiles.cluster;
        if (plan.walk) {
            const int e = dtype == GLA_BF16
                              ? launch_short<__nv_bfloat16>(a, backward, vec4, stream)
                              : launch_short<float>(a, backward, vec4, stream);
            if (e != 0) return GLA_ERR_LAUNCH;
            continue;
        }
        const int e = dtype == GLA_BF16 ? launch_for<__nv_bfloat16>(a, backward, way, stream)
                                        : launch_for<float>(a, backward, way, stream);
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
    const int size = dtype == GLA_BF16 ? 2 : 4;
    if (mixed(h, 4, x, size, n) || mixed(h, 4, log_alpha, 4, n) || mixed(out, size, x, size, n) ||
        mixed(out, size, log_alpha, 4, n) || mixed(out, size, h, 4, n))
        return GLA_ERR_ARG;
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
