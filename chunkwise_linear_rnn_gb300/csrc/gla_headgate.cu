// gla_headgate.cu — prompts through the recurrence with one gate per token and head:
//     S_t = a_t S_{t-1} + k_t^T v_t,     o_t = scale q_t S_t,    a_t = exp(log_alpha_t),
// over a packed batch, token-major, with fewer key heads than value heads.
//
// By chunks of 128 tokens on the tensor cores.  With G_t = log2(a_1 ... a_t) inside a chunk that
// the state S enters, and n its last token,
//     o_t = scale 2^G_t (q_t S + sum_{i <= t} (q_t . k_i) 2^-G_i v_i),
//     S'  = 2^G_n S + sum_i k_i^T (2^(G_n - G_i) v_i).
// One gate a token leaves q, k and v the bf16 numbers that they are: the decays go on the
// scores, on the rows of the output and on v's rows.  A chunk whose gates fall below 2^-60 in
// all takes its rows relative to R_t = max(G_t, -60) instead of G_t, with 2^(G_t - R_t - G_i) on
// the scores, so that nothing overflows; the state's part of rows below is then 2^-60 of its
// size or less where it should be less still.
//
// What is rounded to bf16: the scores and the copy of the state that q multiplies, once for
// each output, as the output itself is.  The state does not lose anything by it: 2^(G_n - G_i) v_i
// enters as the sum of three bf16 numbers, which hold all 24 bits of it, and S' is summed in
// fp32 registers.
//
// One block takes 64 columns of v of one head of a sequence (or of a segment of it) and walks
// its chunks:
//   warps 0-3   state: thread i holds row i of S; adds the chunk's sum, writes the bf16 copy; then
//               the outputs of row i of the chunk
//   warps 4-7   scores: thread t reads row t of Q K^T, decays and masks it, leaves it in TMEM
//   warps 8-11  values: thread t writes row t of the decayed V in three parts
//   warp 12     queues the next tiles by TMA
//   warp 13     sums the chunk's gates
//   warp 14     issues every product
// Products of chunk u, in this order, and when they may start:
//   K^T [V'1 | V'2 | V'3]   the parts are written, the last chunk's sum is read
//   Q S                     the copy of S is written, the last chunk's outputs are read
//   P V, onto Q S           the scores are written
//   Q K^T of chunk u + 1    its tiles are there, chunk u - 1 is done
// so that every warp has the time of the other products for its part.
//
// Long sequences in small numbers are cut into segments: a first launch walks all but the last
// one from a state of zero (k and v alone), and each segment then starts from the states before
// it, S = 2^G S + S_segment.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <new>
#include <vector>

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

void headgate_inputs(Span (&in)[4], const void *q, const void *k, const void *v,
                     const float *log_alpha, int rows, int Hk, int H, int dk, int dv, int size,
                     const gla_headgate_layout &lay) {
    const auto reach = [&](long long st, long long sh, int heads, int d) {
        return rows > 0 ? static_cast<unsigned long long>((rows - 1) * st + (heads - 1) * sh + d) : 0;
    };
    in[0] = span_of(q, reach(lay.q_st, lay.q_sh, Hk, dk), size);
    in[1] = span_of(k, reach(lay.k_st, lay.k_sh, Hk, dk), size);
    in[2] = span_of(v, reach(lay.v_st, lay.v_sh, H, dv), size);
    in[3] = span_of(log_alpha, reach(lay.a_st, lay.a_sh, H, 1), 4);
}

namespace {

constexpr int C = 128;                   // tokens of a chunk
constexpr int kCols = 64;                // columns of v of a block
constexpr int kThreads = 480;
constexpr int kItems = 200;              // segments of one launch: their table is a parameter
constexpr float kFloor = -60.f;          // of R_t
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kBlk = C * 128;       // a tile of 128 rows of 64 bf16

struct Smem {
    // the loaded tiles of a chunk, twice: Q and K by blocks of 64 channels, V
    static constexpr uint32_t kQ = 0, kK = 2 * kBlk, kV = 4 * kBlk, kStage = 5 * kBlk;
    static constexpr uint32_t kW = 2 * kStage;            // the three parts of the decayed V
    static constexpr uint32_t kS = kW + 3 * kBlk;         // bf16 copy of the state
    static constexpr uint32_t kGates = kS + kBlk;         // twice
    static constexpr uint32_t kBar = kGates + 2 * 1040;
    static constexpr uint32_t kSlot = kBar + 256;
    static constexpr uint32_t kBytes = kSlot + 16;
};
static_assert(Smem::kBytes <= 227 * 1024, "shared memory of one block");

// What the gates of a chunk come to: for the scores, by token, 2^-G_i, or -G_i in a chunk that
// falls below the floor (`deep`); the decay from each token to the chunk's end; over all of it,
// and its logarithm.
struct Gates {
    float e[C], w[C];
    float all, total;
    int deep, pad;
};
static_assert(sizeof(Gates) == 1040, "room in Smem");

// Barriers; those of two are taken in turn, chunk u the (u & 1)th.
constexpr int kFull = 0;       // [2] Q and K loaded
constexpr int kFullV = 2;      // [2] V loaded
constexpr int kDone = 4;       // [2] every product of the chunk done: V free, outputs there
constexpr int kGFull = 6;      // [2] gates written
constexpr int kGFree = 8;      // [2] gates read by all
constexpr int kScore = 10;     // [2] Q K^T done
constexpr int kP = 12;         // [2] scores written
constexpr int kParts = 14;     // parts of the decayed V written
constexpr int kSum = 15;       // the chunk's sum done: K and the parts free
constexpr int kSumFree = 16;   // the sum read
constexpr int kCopy = 17;      // copy of the state written
constexpr int kQS = 18;        // Q S done: Q and the copy free
constexpr int kOFree = 19;     // outputs read
constexpr int kDrain = 20;
constexpr int kBars = 21;
static_assert(kBars * 8 <= 256, "room in Smem");

// A segment of a sequence.
struct Item {
    int row, rows;             // first token, tokens
    int n;                     // sequence
    int slot, seg, parts;      // scratch: the sequence's first slot; number of segment, of how many
};

struct Args {
    CUtensorMap tq, tk, tv;
    const float *la, *h0;
    __nv_bfloat16 *o;
    float *hT;
    float *seg_state;          // [slots][H][dk][dv]
    float *seg_log;            // [slots][H]
    long long a_st, a_sh;
    float scale;
    int H, share, dk, dv, tiles;
    int q_step, k_step, v_step;   // from head to head of the tensor maps: 1, or 0 for a shared one
    int wide_store;            // rows of o lie at multiples of 32 bytes
    unsigned int *status;
    Item items[kItems];
};

// TMEM columns: two buffers of scores (Q K^T in fp32, the decayed scores over it), the chunk's
// sum in its three parts, the outputs.
constexpr uint32_t kTScore = 0, kTSum = 256, kTOut = 448;

// Four consecutive tokens' gates of a chunk of n tokens, by lane.
__device__ __forceinline__ void load_gates(const Args &p, long long row, int n, int h, float (&g)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = 4 * lane + j;
        g[j] = i < n ? __ldg(p.la + (row + i) * p.a_st + h * p.a_sh) : 0.f;
    }
}

template <bool STATE>
__device__ __forceinline__ void write_gates(float (&g)[4], Gates &out) {
    const int lane = threadIdx.x & 31;
    // exp(-111) is 0 in 32 bits: a gate of 0 takes part in the sums as this
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (g[j] < -111.f) g[j] = -111.f;
    const float p[4] = {g[0], g[0] + g[1], g[0] + g[1] + g[2], (g[0] + g[1]) + (g[2] + g[3])};
    // sums of the lanes before and behind, each by additions alone: small sums stay exact
    float before = p[3], behind = p[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, before, o);
        const float b = __shfl_down_sync(0xffffffffu, behind, o);
        if (lane >= o) before += a;
        if (lane + o < 32) behind += b;
    }
    const float total = __shfl_sync(0xffffffffu, before, 31);
    before = __shfl_up_sync(0xffffffffu, before, 1);
    behind = __shfl_down_sync(0xffffffffu, behind, 1);
    if (lane == 0) before = 0.f;
    if (lane == 31) behind = 0.f;
    const bool deep = total * kLog2e < kFloor;
    if (!STATE) {
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = -kLog2e * (before + p[j]);
            if (!deep) e[j] = ex2f(e[j]);
        }
        *reinterpret_cast<float4 *>(out.e + 4 * lane) = make_float4(e[0], e[1], e[2], e[3]);
    }
    *reinterpret_cast<float4 *>(out.w + 4 * lane) =
        make_float4(exp_centred(behind + (g[1] + (g[2] + g[3]))), exp_centred(behind + (g[2] + g[3])),
                    exp_centred(behind + g[3]), exp_centred(behind));
    if (lane == 0) {
        out.all = exp_centred(total);
        out.total = total;
        out.deep = deep;
    }
}

// Two fp32 values, for operations on both in one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(uint32_t a, uint32_t b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ Pair pair_of(float a, float b) {
    return pair_of(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ float2 both(Pair r) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t narrow(Pair p) {
    const float2 v = both(p);
    return pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ Pair widen(uint32_t w) { return pair_of(w << 16, w & 0xffff0000u); }

// A pair of values as three pairs of bf16 numbers that add up to it.
__device__ __forceinline__ void split3(Pair x, uint32_t (&part)[3]) {
    const Pair minus = pair_of(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        part[i] = narrow(x);
        if (i < 2) x = fma2(widen(part[i]), minus, x);
    }
}

// Where 16 bytes of row `row` of a tile lie: column group c8 of 8.
__device__ __forceinline__ uint32_t at_tile(int row, int c8) {
    return static_cast<uint32_t>(row) * 128u + (static_cast<uint32_t>(c8 ^ (row & 7)) << 4);
}

__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// STATE: the first launch of divided sequences, whose segments' sums alone are wanted.
template <bool STATE>
__global__ void __launch_bounds__(kThreads, 1) headgate_chunk_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Smem::kBar);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + Smem::kSlot);
    Gates *gates = reinterpret_cast<Gates *>(sm + Smem::kGates);
    const int tile = blockIdx.x % p.tiles, h = blockIdx.x / p.tiles % p.H;
    const Item &it = p.items[blockIdx.x / p.tiles / p.H];
    const int hk = h / p.share, c0 = tile * kCols, dk = p.dk;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the same in a warp, to the compiler too
    const int nch = (it.rows + C - 1) / C;
    const int kblocks = dk > 64 ? 2 : 1, ksteps = (dk + 15) / 16;
    const uint32_t a0 = smem_u32(sm);
    unsigned int *status = p.status;

    if (warp == 0) tmem_alloc(slot, 512);
    if (tid == 32) {
        for (int i = 0; i < kBars; ++i) {
            const bool by_warps = i == kP || i == kP + 1 || i == kParts || i == kSumFree ||
                                  i == kCopy || i == kOFree;
            const bool by_all = i == kGFree || i == kGFree + 1;
            mbar_init(&bar[i], by_all ? (STATE ? 8 : 12) : by_warps ? 4 : 1);
        }
        fence_mbar_init();
    }
    // channels past the first block: rows of the state that stay 0
    if (kblocks == 1)
        for (uint32_t i = tid * 16; i < kBlk; i += kThreads * 16)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                *reinterpret_cast<uint4 *>(sm + s * Smem::kStage + Smem::kK + kBlk + i) =
                    make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;   // the warp's lanes
    // a warp's wait for the barrier's phase of chunk u (of two in turn, or one)
    auto wait2 = [&](int b, int u) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(&bar[b + (u & 1)],
                                                         static_cast<uint32_t>(u >> 1) & 1u, status));
    };
    auto wait1 = [&](int b, int u) {
        return __all_sync(0xffffffffu,
                          mbar_wait_bounded(&bar[b], static_cast<uint32_t>(u) & 1u, status));
    };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[b]);
    };

    if (warp < 4) {
        // ================================================================ state
        const int i = tid;
        Pair S[kCols / 2];
        auto clear = [&]() {
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) S[c] = 0;
        };
        clear();
        auto state_row = [&](long long entry) {   // of [.][H][dk][dv]
            return ((entry * p.H + h) * dk + i) * p.dv + c0;
        };
        auto add_row = [&](const float *from, float a) {
            if (i >= dk) return;
            const Pair aa = pair_of(a, a);
#pragma unroll
            for (int c = 0; c < kCols; c += 4)
                if (c0 + c < p.dv) {
                    const float4 x = *reinterpret_cast<const float4 *>(from + c);
                    S[c / 2] = fma2(aa, S[c / 2], pair_of(x.x, x.y));
                    S[c / 2 + 1] = fma2(aa, S[c / 2 + 1], pair_of(x.z, x.w));
                }
        };
        auto put_row = [&](float *to) {
            if (i >= dk) return;
#pragma unroll
            for (int c = 0; c < kCols; c += 4)
                if (c0 + c < p.dv) {
                    const float2 x = both(S[c / 2]), y = both(S[c / 2 + 1]);
                    *reinterpret_cast<float4 *>(to + c) = make_float4(x.x, x.y, y.x, y.y);
                }
        };
        auto put_copy = [&]() {
#pragma unroll
            for (int c = 0; c < kCols / 8; ++c)
                *reinterpret_cast<uint4 *>(sm + Smem::kS + at_tile(i, c)) =
                    make_uint4(narrow(S[4 * c]), narrow(S[4 * c + 1]), narrow(S[4 * c + 2]),
                               narrow(S[4 * c + 3]));
            fence_proxy_async_smem();
            arrive(kCopy);
        };
        if (STATE) {
            // h0 is kept for the second launch, whose blocks may write hT over it
            if (it.seg == 0 && p.h0) {
                add_row(p.h0 + state_row(it.n), 0.f);
                put_row(p.seg_state + state_row(it.slot + it.parts - 1));
                clear();
            }
        } else {
            if (p.h0)
                add_row(it.parts > 1 ? p.seg_state + state_row(it.slot + it.parts - 1)
                                     : p.h0 + state_row(it.n), 0.f);
            for (int m = 0; m < it.seg; ++m)
                add_row(p.seg_state + state_row(it.slot + m),
                        exp_centred(p.seg_log[static_cast<long long>(it.slot + m) * p.H + h]));
            if (nch > 0) put_copy();
        }
        float total = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
            if (!(ok = wait2(kGFull, u))) break;
            const Gates &g = gates[u & 1];
            const Pair a = pair_of(g.all, g.all);
            const float f =
                STATE ? 0.f : p.scale * (g.deep ? ex2f(fmaxf(-g.e[i], kFloor)) : 1.f / g.e[i]);
            const Pair ff = pair_of(f, f);
            if (STATE) total += g.total;
            arrive(kGFree + (u & 1));
            if (!(ok = wait1(kSum, u))) break;
            tc_fence_after();
            // the next 8 columns are on their way while these are added
            uint32_t x[2][3][8];
            auto fetch = [&](int c) {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    tmem_ld8(tmem + lanes + kTSum + i * kCols + c, x[c / 8 & 1][i]);
            };
            fetch(0);
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
                tmem_wait_ld();
                if (c + 8 < kCols) fetch(c + 8);
                const uint32_t(&now)[3][8] = x[c / 8 & 1];
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    S[(c + j) / 2] = fma2(a, S[(c + j) / 2],
                                          add2(pair_of(now[0][j], now[0][j + 1]),
                                               add2(pair_of(now[1][j], now[1][j + 1]),
                                                    pair_of(now[2][j], now[2][j + 1]))));
            }
            tc_fence_before();
            arrive(kSumFree);
            if (STATE) continue;
            if (u + 1 < nch) {
                if (!(ok = wait1(kQS, u))) break;
                put_copy();
            }
            // the outputs of row t = i
            const int left = u * C + i < it.rows ? p.dv - c0 : 0;
            __nv_bfloat16 *to =
                p.o + (static_cast<long long>(it.row + u * C + i) * p.H + h) * p.dv + c0;
            if (!(ok = wait2(kDone, u))) break;
            tc_fence_after();
            uint32_t r[2][16];
            tmem_ld16(tmem + lanes + kTOut, r[0]);
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
                tmem_wait_ld();
                if (c + 16 < kCols) {
                    tmem_ld16(tmem + lanes + kTOut + c + 16, r[c / 16 + 1 & 1]);
                } else {
                    tc_fence_before();
                    arrive(kOFree);
                }
                uint32_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = narrow(mul2(ff, pair_of(r[c / 16 & 1][2 * j], r[c / 16 & 1][2 * j + 1])));
                if (p.wide_store) {
                    if (c < left) store32(to + c, v);
                } else {
                    if (c < left)
                        *reinterpret_cast<uint4 *>(to + c) = make_uint4(v[0], v[1], v[2], v[3]);
                    if (c + 8 < left)
                        *reinterpret_cast<uint4 *>(to + c + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                }
            }
        }
        if (ok) {
            if (STATE) {
                put_row(p.seg_state + state_row(it.slot + it.seg));
                if (tid == 0 && tile == 0)
                    p.seg_log[static_cast<long long>(it.slot + it.seg) * p.H + h] = total;
            } else if (p.hT && it.seg == it.parts - 1) {
                put_row(p.hT + state_row(it.n));
            }
        }
    } else if (warp < 8) {
        // ================================================================ scores
        const int w = warp - 4, t = tid - 128;
#pragma unroll 1
        for (int u = 0; !STATE && u < nch; ++u) {
            if (!(wait2(kGFull, u) && wait2(kScore, u))) break;
            tc_fence_after();
            const Gates &g = gates[u & 1];
            const uint32_t at = tmem + lanes + kTScore + (u & 1) * C;
            const float4 *e4 = reinterpret_cast<const float4 *>(g.e);
            const bool deep = g.deep;
            const float base = deep ? -g.e[t] - fmaxf(-g.e[t], kFloor) : 0.f;
            uint32_t out[16];
            // the tokens of warps before this one's, then its own, then those behind
#pragma unroll 1
            for (int b = 0; b <= w; ++b) {
                uint32_t r[32];
                float4 e[8];
                tmem_ld32(at + 32 * b, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = e4[8 * b + j];
                tmem_wait_ld();
                if (b == w) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j > lane) r[j] = 0u;
                }
                if (!deep) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 f = e[j / 4];
                        out[j / 2] = narrow(mul2(pair_of(r[j], r[j + 1]), pair_of(f.x, f.y)));
                        out[j / 2 + 1] = narrow(mul2(pair_of(r[j + 2], r[j + 3]), pair_of(f.z, f.w)));
                    }
                } else {
                    // 2^(base - G_i) of a later token may be infinite: a masked score stays 0
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float f0 = j % 4 ? e[j / 4].z : e[j / 4].x;
                        const float f1 = j % 4 ? e[j / 4].w : e[j / 4].y;
                        const int i = 32 * b + j;
                        out[j / 2] = pack_bf16x2(
                            i <= t ? __uint_as_float(r[j]) * ex2f(base + f0) : 0.f,
                            i + 1 <= t ? __uint_as_float(r[j + 1]) * ex2f(base + f1) : 0.f);
                    }
                }
                tmem_st16(at + 16 * b, out);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) out[j] = 0u;
#pragma unroll 1
            for (int b = w + 1; b < 4; ++b) tmem_st16(at + 16 * b, out);
            tmem_wait_st();
            tc_fence_before();
            arrive(kP + (u & 1));
            arrive(kGFree + (u & 1));
        }
    } else if (warp < 12) {
        // ================================================================ values
        const int t = tid - 256;
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
            const bool short_chunk = it.rows - u * C < C;   // whose rows of K are cleared too
            if (!(wait2(kFullV, u) && (!short_chunk || wait2(kFull, u)) && wait2(kGFull, u) &&
                  (u == 0 || wait1(kSum, u - 1))))
                break;
            uint8_t *st = sm + (u & 1) * Smem::kStage;
            const float w = gates[u & 1].w[t];
            const Pair f = pair_of(w, w);
            const bool real = u * C + t < it.rows;
            // half a row's loads before the first store, which the compiler has to keep in order
#pragma unroll 1
            for (int c0 = 0; c0 < kCols / 8; c0 += 4) {
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint8_t *at = st + Smem::kV + at_tile(t, c0 + c);
                    v[c] = *reinterpret_cast<const uint4 *>(at);
                    if (!real) {
                        // the next sequence's rows, which may hold anything: no part of any product
                        v[c] = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(at) = v[c];
                        at += Smem::kK - Smem::kV;
                        *reinterpret_cast<uint4 *>(at) = v[c];
                        if (kblocks == 2) *reinterpret_cast<uint4 *>(at + kBlk) = v[c];
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t part[4][3];
                    split3(mul2(f, widen(v[c].x)), part[0]);
                    split3(mul2(f, widen(v[c].y)), part[1]);
                    split3(mul2(f, widen(v[c].z)), part[2]);
                    split3(mul2(f, widen(v[c].w)), part[3]);
                    uint8_t *to = sm + Smem::kW + at_tile(t, c0 + c);
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        *reinterpret_cast<uint4 *>(to + i * kBlk) =
                            make_uint4(part[0][i], part[1][i], part[2][i], part[3][i]);
                }
            }
            fence_proxy_async_smem();
            arrive(kParts);
            arrive(kGFree + (u & 1));
        }
    } else if (warp == 12) {
        // ================================================================ loads
        int loads = 0;
        auto load_k = [&](int u) {
            uint64_t *full = &bar[kFull + (u & 1)];
            warp_expect_tx(full, kblocks * (STATE ? 1 : 2) * kBlk);
            for (int b = 0; b < kblocks; ++b)
                warp_tma_load_3d(sm + (u & 1) * Smem::kStage + Smem::kK + b * kBlk, &p.tk, full,
                                 b * 64, hk * p.k_step, it.row + u * C);
            loads = u + 1;
        };
        auto load_q = [&](int u) {
            for (int b = 0; !STATE && b < kblocks; ++b)
                warp_tma_load_3d(sm + (u & 1) * Smem::kStage + Smem::kQ + b * kBlk, &p.tq,
                                 &bar[kFull + (u & 1)], b * 64, hk * p.q_step, it.row + u * C);
        };
        auto load_v = [&](int u) {
            uint64_t *full = &bar[kFullV + (u & 1)];
            warp_expect_tx(full, kBlk);
            warp_tma_load_3d(sm + (u & 1) * Smem::kStage + Smem::kV, &p.tv, full, c0,
                             h * p.v_step, it.row + u * C);
        };
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
            // each tile as soon as its last product of chunk u - 2 is done
            if (u >= 2 && !wait1(kSum, u - 2)) break;
            load_k(u);
            if (!STATE && u >= 2 && !wait1(kQS, u - 2)) break;
            load_q(u);
            if (u >= 2 && !wait2(kDone, u - 2)) break;
            load_v(u);
        }
        // loads that an expired wait left under way land before the block gives up its memory
        for (int u = max(0, loads - 2); u < loads; ++u) wait2(kFull, u), wait2(kFullV, u);
    } else if (warp == 13) {
        // ================================================================ gates
        float g[4], next[4];
        if (nch > 0) load_gates(p, it.row, min(C, it.rows), h, next);
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = next[j];
            if (u + 1 < nch)
                load_gates(p, it.row + (u + 1) * C, min(C, it.rows - (u + 1) * C), h, next);
            if (u >= 2 && !wait2(kGFree, u - 2)) break;
            write_gates<STATE>(g, gates[u & 1]);
            arrive(kGFull + (u & 1));
        }
    } else {
        // ================================================================ products
        // a step of 16 of the common dimension, in descriptors: 16 rows of a tile whose rows are
        // that dimension, 32 bytes of a row (and on to the next tile of 64 after four) otherwise
        constexpr uint64_t kRows = 2048 >> 4, kBytes32 = 32 >> 4, kNext = (kBlk - 96) >> 4;
        auto scores = [&](int u) {
            constexpr uint32_t id = idesc_bf16(C, C, false, false);   // Q [t][c], K [i][c]
            const uint32_t st = a0 + (u & 1) * Smem::kStage;
            uint64_t q = sw128_desc(st + Smem::kQ, 16, 1024), k = sw128_desc(st + Smem::kK, 16, 1024);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < ksteps; ++i) {
                warp_mma_bf16_ss(tmem + kTScore + (u & 1) * C, q, k, id, i > 0);
                const uint64_t on = (i & 3) == 3 ? kNext : kBytes32;
                q += on;
                k += on;
            }
            warp_mma_commit(&bar[kScore + (u & 1)]);
        };
        if (!STATE && nch > 0 && wait2(kFull, 0)) scores(0);
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
            const uint32_t st = a0 + (u & 1) * Smem::kStage;
            if (!(wait2(kFull, u) && wait1(kParts, u) && (u == 0 || wait1(kSumFree, u - 1)))) break;
            tc_fence_after();
            // K^T [c][t] by the parts [t][3 x 64]
            constexpr uint32_t id_sum = idesc_bf16(128, 3 * kCols, true, true);
            uint64_t x = sw128_desc(st + Smem::kK, kBlk, 1024);
            uint64_t y = sw128_desc(a0 + Smem::kW, kBlk, 1024);
#pragma unroll 1
            for (int i = 0; i < C / 16; ++i, x += kRows, y += kRows)
                warp_mma_bf16_ss(tmem + kTSum, x, y, id_sum, i > 0);
            warp_mma_commit(&bar[kSum]);
            if (STATE) {
                warp_mma_commit(&bar[kDone + (u & 1)]);
                continue;
            }
            if (!(wait1(kCopy, u) && (u == 0 || wait1(kOFree, u - 1)))) break;
            tc_fence_after();
            // Q [t][c] by S [c][64]
            constexpr uint32_t id_out = idesc_bf16(C, kCols, false, true);
            x = sw128_desc(st + Smem::kQ, 16, 1024);
            y = sw128_desc(a0 + Smem::kS, kBlk, 1024);
#pragma unroll 1
            for (int i = 0; i < ksteps; ++i, y += kRows) {
                warp_mma_bf16_ss(tmem + kTOut, x, y, id_out, i > 0);
                x += (i & 3) == 3 ? kNext : kBytes32;
            }
            warp_mma_commit(&bar[kQS]);
            if (!wait2(kP, u)) break;
            tc_fence_after();
            // P [t][i] by V [i][64], onto Q S
            y = sw128_desc(st + Smem::kV, kBlk, 1024);
            uint32_t score = tmem + kTScore + (u & 1) * C;
#pragma unroll 1
            for (int i = 0; i < C / 16; ++i, y += kRows, score += 8)
                warp_mma_bf16_ts(tmem + kTOut, score, y, id_out, 1u);
            warp_mma_commit(&bar[kDone + (u & 1)]);
            if (u + 1 < nch) {
                // the scores of chunk u - 1 lay where these go
                if (!(wait2(kFull, u + 1) && (u == 0 || wait2(kDone, u - 1)))) break;
                scores(u + 1);
            }
        }
        // every product ends before TMEM and shared memory are given up
        warp_mma_commit(&bar[kDrain]);
        wait1(kDrain, 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- the plan

// How the sequences are cut: chunks of a segment, at most (INT_MAX: none is cut), and slots of
// scratch.
struct Plan {
    int most;
    long long slots;
};

int chunks_of(const int *cu, int n) { return (cu[n + 1] - cu[n] + C - 1) / C; }
int parts_of(int chunks, int most) { return chunks > most ? (chunks + most - 1) / most : 1; }

// The blocks of all heads and column tiles run in rounds on the SMs; a launch takes at least its
// longest segment, and at least its share of all chunks.  Cutting costs a launch that walks all
// but the last segments for their sums (kSumCost of a chunk's whole work each) and what it takes
// to begin.  Of one cut and of 2 to 32 parts for the longest sequence, the one that this says
// is the quickest.
Plan make_plan(const int *cu, int N, int H, int dv) {
    constexpr double kSms = 152, kSumCost = 0.5, kBegin = 4;
    const double lanes = static_cast<double>(H) * ((dv + kCols - 1) / kCols) / kSms;
    int longest = 0;
    long long all = 0;
    for (int n = 0; n < N; ++n) {
        longest = std::max(longest, chunks_of(cu, n));
        all += chunks_of(cu, n);
    }
    Plan best = {INT_MAX, 0};
    double least = std::max<double>(longest, all * lanes);
    for (int k = 2; k <= 32 && k <= longest; ++k) {
        const int most = (longest + k - 1) / k;
        const double whole = std::max<double>(most, all * lanes);
        if (whole + kBegin >= least) continue;   // not even with the first launch for nothing
        long long first = 0, slots = 0;
        for (int n = 0; n < N; ++n) {
            const int c = chunks_of(cu, n), parts = parts_of(c, most);
            if (parts == 1) continue;
            first += c - c / parts;
            slots += parts;
        }
        const double cost = whole + kBegin + kSumCost * std::max<double>(most, first * lanes);
        if (cost < least) {
            least = cost;
            best = {most, slots};
        }
    }
    return best;
}

size_t scratch_of(const Plan &plan, int H, int dk, int dv) {
    return static_cast<size_t>(plan.slots) * H * (static_cast<size_t>(dk) * dv + 4) * sizeof(float);
}

bool bounds_ok(const int *cu, int N, int T) {
    if (!cu || N <= 0 || T < 0 || cu[0] != 0 || cu[N] != T) return false;
    for (int n = 0; n < N; ++n)
        if (cu[n + 1] < cu[n]) return false;
    return true;
}

template <bool STATE>
bool prepared() {
    // the attribute belongs to the device's copy of the function
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(headgate_chunk_kernel<STATE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(Smem::kBytes)) != cudaSuccess)
        return false;
    done[dev].store(true, std::memory_order_release);
    return true;
}

template <bool STATE>
bool launch(Args &a, const std::vector<Item> &items, cudaStream_t stream) {
    if (items.empty()) return true;
    if (!prepared<STATE>()) return false;
    for (size_t first = 0; first < items.size(); first += kItems) {
        const size_t n = std::min<size_t>(kItems, items.size() - first);
        std::copy(items.begin() + first, items.begin() + first + n, a.items);
        const unsigned grid = static_cast<unsigned>(n) * a.H * a.tiles;
        headgate_chunk_kernel<STATE><<<grid, kThreads, Smem::kBytes, stream>>>(a);
        if (cudaGetLastError() != cudaSuccess) return false;
    }
    return true;
}

int run(Args &a, const int *cu, int N, const Plan &plan, cudaStream_t stream) {
    std::vector<Item> whole, sums;
    int slot = 0;
    for (int n = 0; n < N; ++n) {
        const int chunks = chunks_of(cu, n), parts = parts_of(chunks, plan.most);
        for (int s = 0, c = 0; s < parts; ++s) {
            const int next = static_cast<int>(static_cast<long long>(chunks) * (s + 1) / parts);
            const int row = cu[n] + c * C, end = s + 1 < parts ? cu[n] + next * C : cu[n + 1];
            const Item it = {row, end - row, n, parts > 1 ? slot : -1, s, parts};
            whole.push_back(it);
            if (s + 1 < parts) sums.push_back(it);
            c = next;
        }
        if (parts > 1) slot += parts;
    }
    // the longest first, so that the last round is short
    auto longer = [](const Item &x, const Item &y) { return x.rows > y.rows; };
    std::stable_sort(whole.begin(), whole.end(), longer);
    std::stable_sort(sums.begin(), sums.end(), longer);
    return launch<true>(a, sums, stream) && launch<false>(a, whole, stream) ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace
}  // namespace gla

extern "C" {

unsigned long gla_headgate_fwd_varlen_scratch(const int *cu_seqlens, int N, int H, int dk, int dv) {
    using namespace gla;
    if (N <= 0 || H <= 0 || dk <= 0 || dv <= 0 || !cu_seqlens ||
        !bounds_ok(cu_seqlens, N, cu_seqlens[N]))
        return 0;
    return scratch_of(make_plan(cu_seqlens, N, H, dv), H, dk, dv);
}

int gla_headgate_fwd_varlen(const void *q, const void *k, const void *v, const float *log_alpha,
                            float scale, const float *h0, void *o, float *hT,
                            const int *cu_seqlens, int N, int T_total, int Hk, int H, int dk,
                            int dv, const gla_headgate_layout *layout, void *scratch,
                            unsigned long scratch_bytes, cudaStream_t stream) {
    using namespace gla;
    if (!layout || !bounds_ok(cu_seqlens, N, T_total)) return GLA_ERR_ARG;
    if (T_total > 0 && (!q || !k || !v || !log_alpha || !o)) return GLA_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(h0) | reinterpret_cast<uintptr_t>(hT) |
         reinterpret_cast<uintptr_t>(scratch)) & 15)
        return GLA_ERR_ARG;
    int st = headgate_check(q, k, v, log_alpha, nullptr, o, Hk, H, dk, dv, *layout);
    if (st != GLA_OK) return st;
    if (T_total > 1 && (!layout->q_st || !layout->k_st || !layout->v_st)) return GLA_ERR_ARG;
    // a chunk's last row is counted on past the last token in 32 bits
    if (T_total > INT_MAX - C) return GLA_ERR_ARG;
    Span in[4];
    headgate_inputs(in, q, k, v, log_alpha, T_total, Hk, H, dk, dv, 2, *layout);
    const unsigned long long states = static_cast<unsigned long long>(N) * H * dk * dv;
    const Span out = span_of(o, static_cast<unsigned long long>(T_total) * H * dv, 2);
    const Span begin = span_of(h0, states, 4), end = span_of(hT, states, 4);
    if (meets_any(out, in) || meets_any(end, in) || meet(out, begin) || meet(out, end) ||
        (h0 != hT && meet(begin, end)))
        return GLA_ERR_ARG;
    const Plan plan = make_plan(cu_seqlens, N, H, dv);
    if (plan.slots > INT_MAX) return GLA_ERR_ARG;
    const size_t need = scratch_of(plan, H, dk, dv);
    if (need > 0 && (!scratch || scratch_bytes < need)) return GLA_ERR_SCRATCH;
    int sms = 0;
    Args a = {};
    st = usable_device(&sms, &a.status);
    if (st != GLA_OK) return st;
    a.la = log_alpha;
    a.h0 = h0;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.hT = hT;
    a.seg_state = static_cast<float *>(scratch);
    a.seg_log = a.seg_state + static_cast<size_t>(plan.slots) * H * dk * dv;
    a.a_st = layout->a_st;
    a.a_sh = layout->a_sh;
    a.scale = scale;
    a.H = H;
    a.share = H / Hk;
    a.dk = dk;
    a.dv = dv;
    a.tiles = (dv + kCols - 1) / kCols;
    a.wide_store = dv % 16 == 0 && (reinterpret_cast<uintptr_t>(o) & 31) == 0;
    if (T_total > 0) {
        const gla_headgate_layout &l = *layout;
        a.q_step = Hk > 1 && l.q_sh;
        a.k_step = Hk > 1 && l.k_sh;
        a.v_step = H > 1 && l.v_sh;
        if (!head_map(&a.tq, q, dk, a.q_step ? Hk : 1, T_total, l.q_sh, l.q_st, C) ||
            !head_map(&a.tk, k, dk, a.k_step ? Hk : 1, T_total, l.k_sh, l.k_st, C) ||
            !head_map(&a.tv, v, dv, a.v_step ? H : 1, T_total, l.v_sh, l.v_st, C))
            return GLA_ERR_LAUNCH;
    }
    try {
        return run(a, cu_seqlens, N, plan, stream);
    } catch (const std::bad_alloc &) {
        return GLA_ERR_ALLOC;
    }
}

}  // extern "C"
