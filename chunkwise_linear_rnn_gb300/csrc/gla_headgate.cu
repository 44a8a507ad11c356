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
// the scores and 2^(G_t - R_t) on q_t S, so that nothing overflows.
//
// What is rounded to bf16: the scores and the copy of the state that q multiplies, once for
// each output, as the output itself is (scores of sequences of one chunk at most enter in two
// parts instead).  The state does not lose anything by it: 2^(G_n - G_i) v_i enters as the sum
// of three bf16 numbers, which hold all 24 bits of it, and S' is summed in fp32 registers.
//
// One block takes 128 columns of v of one head of a sequence (or of a segment of it) and walks
// its chunks:
//   warps 0-7   values and state.  Of the decayed V, transposed on its way from shared memory, each
//               warp writes 32 columns of 64 tokens to TMEM, part by part; of the state, thread
//               (column, half) holds 64 channels, adds the chunk's sum and writes the bf16 copy
//   warps 8-11  scores and outputs: thread t reads row t of Q K^T, decays and masks it, leaves it
//               in TMEM; later it stores row t of the outputs
//   warp 12     queues the next tiles by TMA
//   warp 13     sums the chunk's gates
//   warp 14     issues every product
// Products of chunk u, in this order, and when they may start:
//   V'1^T K            the first part is written, the last chunk's sum is read
//   Q K^T              chunk u - 1 is done
//   Q S                the copy of S is written, the last chunk's outputs are read
//   V'2^T K, V'3^T K   onto the first; their parts are written (two slots take turns)
//   P V, onto Q S      the scores are written, and in a chunk below the floor Q S is scaled
// Q S comes early so that one tile of Q is enough, which leaves room for a third one of V.
//
// HBM's floor for 16,384 tokens, 16 heads of 128 and 128 is 41 us (278 MB); measured on one GB300
// 60 us (0.68), with 128 of 152 SMs in use.  Of about 6,000 cycles a chunk its products take 3,120,
// shared memory's traffic 3,328 (416 KB at 128 bytes a cycle), the warps' instructions about 3,000
// issue slots of a scheduler.  On the SMs in use the tensor pipe and L1 with shared memory are busy
// for 51 % of the launch, issue slots for 48 %: what is left is the chain from warp to warp.
// On an earlier form of this kernel, 60.1 us with two tiles of V, it took 12 % less without the
// values' splitting, 13 % without the outputs' stores, 2 to 4 % without the work on states,
// scores or copies.  Measured beside the next one (58 us), same case: parts of V' in shared memory
// and 64 columns a block, 78 us; outputs through shared memory and TMA stores, 60; all outputs
// read before the first store, 67; the next chunk's tiles pulled into L2 ahead of time, 60 to
// 63; the same products issued by one lane alone (180-240 cycles each), 113 for 94 in the form
// with 64 columns.  The decays in two numbers, what of Q S is left below the floor and scores
// in two parts by sequence took that to 60.
//
// A block has an SM to itself, so blocks run in rounds: 9 such prompts of 2,048 tokens take 65 us, 10
// take 111, 19 take 121.  Where v has 64 columns or fewer, half of a block's columns are empty:
// 8 + 16 heads of 128 x 64 take 54 us for the 63 of 128 x 128.
//
// Long sequences in small numbers are cut into segments: a first launch walks all but the last
// one from a state of zero (k and v alone), and each segment then starts from the states before
// it, S = 2^G S + S_segment.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>
#include <vector>

#include "gla.h"
#include "gla_exp.cuh"
#include "gla_internal.h"
#include "gla_ptx_warp.cuh"

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
constexpr int kCols = 128;               // columns of v of a block
constexpr int kThreads = 512;
constexpr int kItems = 200;              // segments of one launch: their table is a parameter
constexpr float kFloor = -60.f;          // of R_t
constexpr float kSteep = -256.f;         // of G_n where sums of 32 bits are enough
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kBlk = C * 128;       // a tile of 128 rows of 64 bf16

struct Smem {
    // the loaded tiles by blocks of 64 channels or columns: Q, K of two chunks, V of three
    static constexpr uint32_t kQ = 0, kK = 2 * kBlk, kV = 6 * kBlk, kTile = 2 * kBlk;
    static constexpr uint32_t kS = 12 * kBlk;            // bf16 copy of the state [column][channel]
    static constexpr uint32_t kGates = kS + 2 * kBlk;     // twice
    static constexpr uint32_t kBar = kGates + 2 * 1296;
    static constexpr uint32_t kSlot = kBar + 288;
    static constexpr uint32_t kBytes = kSlot + 16;
};
static_assert(Smem::kBytes <= 227 * 1024, "shared memory of one block");

// What the gates of a chunk come to: for the scores, by token, 2^-G_i, or -G_i in a chunk that
// falls below the floor (`deep`); the decay from each token to the chunk's end; over all of it, and
// its logarithm.
// Behind many steep gates |G| is up to 24,000, where sums of 32 bits are 2^-7 off.  Chunks that fall
// below kSteep have it as e_i + rest_i, summed in 64 bits, 2^-18 off.  Above it the eight additions
// in 32 bits are 2^-14 off at worst, far less than the scores' rounding, and quicker (8 prompts of 2,048
// tokens 58.0 us for 59.9, the ragged ones 122 for 127); scores in two parts take the first form
// below the floor already.
struct Gates {
    float e[C], w[C];
    uint32_t rest[C / 2];
    float all, total;
    int deep, steep;
};
static_assert(sizeof(Gates) == 1296, "room in Smem");

// Barriers; those of two are taken in turn: chunk u the (u & 1)th, part j = 3 u + i by slots.  A
// wait names its phase by parity alone, so the next phase of its barrier must need something that
// comes after the wait.  The loads' wait for a chunk's sum is why kSum has two though there is one
// sum: the next chunk's needs nothing that they queue behind it, the one after that does.
constexpr int kFull = 0;       // [2] K loaded
constexpr int kDone = 4;       // [2] outputs there, V free (not for sums alone)
constexpr int kGFull = 6;      // [2] gates written
constexpr int kGFree = 8;      // [2] gates read by all
constexpr int kScore = 10;     // Q K^T done
constexpr int kP = 11;         // scores written
constexpr int kSum = 12;       // [2] the chunk's sum done, K free; for sums alone V too
constexpr int kSumFree = 14;   // [sums] the sum read
constexpr int kCopy = 16;      // copy of the state written
constexpr int kQS = 17;        // Q S done: Q and the copy free
constexpr int kOFree = 18;     // outputs read
constexpr int kDrain = 19;
constexpr int kFullV = 22;     // [3] V loaded; chunk u the (u % 3)th
constexpr int kFullQ = 2;      // Q loaded
constexpr int kPart = 25;      // [slots] part of the decayed V written
constexpr int kPartFree = 29;  // [slots] its product done
constexpr int kBars = 33;
static_assert(kBars * 8 <= 288, "room in Smem");

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

// TMEM columns: the scores (Q K^T in fp32, the decayed scores over it), two slots for parts of V',
// the chunk's sum, the outputs.
constexpr uint32_t kTScore = 0, kTPart = 128, kTSum = 256, kTOut = 384;
// The sums alone leave room for four slots and two sums.
template <bool STATE>
struct Turns {
    static constexpr int kSlots = STATE ? 4 : 2, kSums = STATE ? 2 : 1;
    __device__ __forceinline__ static uint32_t part(int j) {
        return (STATE ? kTScore : kTPart) + j % kSlots * 64;
    }
    __device__ __forceinline__ static uint32_t sum(int u) { return kTSum + u % kSums * 128; }
};

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
__device__ __forceinline__ void write_gates(float (&g)[4], Gates &out, bool fine) {
    const int lane = threadIdx.x & 31;
    // exp(-130) is 0 in 32 bits, 2^60 of it too: a gate of 0 takes part in the sums as this
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (g[j] < -130.f) g[j] = -130.f;
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
    const bool deep = total * kLog2e < kFloor, steep = fine ? deep : total * kLog2e < kSteep;
    if (!STATE) {
        float e[4];
        if (!steep) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                e[j] = -kLog2e * (before + p[j]);
                if (!deep) e[j] = ex2f(e[j]);
            }
        } else {
            double own[4], sum = 0.;
#pragma unroll
            for (int j = 0; j < 4; ++j) own[j] = sum += g[j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double a = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += a;
            }
            sum -= own[3];
            float rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double x = -1.4426950408889634 * (sum + own[j]);
                e[j] = static_cast<float>(x);
                rest[j] = static_cast<float>(x - e[j]);
            }
            *reinterpret_cast<uint2 *>(out.rest + 2 * lane) =
                make_uint2(pack_bf16x2(rest[0], rest[1]), pack_bf16x2(rest[2], rest[3]));
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
        out.steep = steep;
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

// What is left of a pair of values after a pair of bf16 numbers.
__device__ __forceinline__ Pair left_of(Pair x, uint32_t part) {
    return fma2(widen(part), pair_of(-1.f, -1.f), x);
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane l gets row l / 4 of each, columns
// 2 (l % 4) and one more.
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// 16 lanes of TMEM from the one in taddr, 32 columns: registers 2 k and 2 k + 1 are such matrices
// of columns 4 k to 4 k + 3, lanes 0-7 and 8-15.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Registers of a thread from here on; a group of four warps together.  The block was launched with
// 128 for each of 512 threads: 2 x 168 + 112 + 64 a group of four.
template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
    const int cblocks = p.dv - c0 > 64 ? 2 : 1;
    const uint32_t a0 = smem_u32(sm);
    unsigned int *status = p.status;
    // A sequence of one chunk at most: all of its outputs are made up of few scores, whose rounding
    // does not average out.  They are taken in two parts, 2^-16 off instead of 2^-8.  This goes by
    // the sequence's own length, so that a short prompt's outputs do not depend on the others of its
    // batch.  (Loops of their own: as a condition in the walk it costs the others 4 %, as a launch of
    // its own 14 us where both kinds are there, this way 1 to 2 %.)
    const bool fine = !STATE && it.parts == 1 && it.rows <= C;

    if (warp == 0) tmem_alloc(slot, 512);
    if (tid == 32) {
        for (int i = 0; i < kBars; ++i) {
            int count = 1;
            if (i == kGFree || i == kGFree + 1) count = STATE ? 8 : 12;
            if ((i >= kPart && i < kPart + 4) || i == kSumFree || i == kSumFree + 1 || i == kCopy)
                count = 8;
            if (i == kP || i == kOFree) count = 4;
            mbar_init(&bar[i], count);
        }
        fence_mbar_init();
    }
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
    auto wait3 = [&](int b, int u) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(&bar[b + u % 3],
                                                         static_cast<uint32_t>(u / 3) & 1u, status));
    };
    using Turn = Turns<STATE>;
    auto wait_part = [&](int b, int j) {
        return __all_sync(0xffffffffu,
                          mbar_wait_bounded(&bar[b + j % Turn::kSlots],
                                            static_cast<uint32_t>(j / Turn::kSlots) & 1u, status));
    };
    auto wait_sum_free = [&](int u) {
        return __all_sync(0xffffffffu,
                          mbar_wait_bounded(&bar[kSumFree + u % Turn::kSums],
                                            static_cast<uint32_t>(u / Turn::kSums) & 1u, status));
    };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[b]);
    };

    if (warp < 8) {
        // ================================================================ values and state
        registers_up<168>();
        const int half = warp >> 2, c = 32 * (warp & 3) + lane;   // of the state: channels, column
        const bool mine = c0 + c < p.dv;
        Pair S[32];
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = 0;
        };
        clear();
        const int rows = min(64, dk - 64 * half);                 // channels there are
        auto state_at = [&](long long entry) {                    // of [.][H][dk][dv]
            return ((entry * p.H + h) * dk + 64 * half) * p.dv + c0 + c;
        };
        auto add_state = [&](const float *from, float a) {
            const Pair aa = pair_of(a, a);
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                float x[32];   // all on their way before the first is added
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = mine && i + j < rows ? __ldcg(from + static_cast<long long>(i + j) * p.dv)
                                                : 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    S[(i + j) / 2] = fma2(aa, S[(i + j) / 2], pair_of(x[j], x[j + 1]));
            }
        };
        auto put_state = [&](float *to) {
#pragma unroll
            for (int i = 0; i < 64; i += 2)
                if (mine && i < rows) {
                    const float2 x = both(S[i / 2]);
                    to[static_cast<long long>(i) * p.dv] = x.x;
                    to[static_cast<long long>(i + 1) * p.dv] = x.y;
                }
        };
        auto put_copy = [&]() {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4 *>(sm + Smem::kS + half * kBlk + at_tile(c, i)) =
                    make_uint4(narrow(S[4 * i]), narrow(S[4 * i + 1]), narrow(S[4 * i + 2]),
                               narrow(S[4 * i + 3]));
            fence_proxy_async_smem();
            arrive(kCopy);
        };
        // this warp's 32 columns of 64 tokens of the decayed V: what the parts so far leave of them
        Pair left[2][16];
        float decay = 0.f, total = 0.f;
        const uint32_t part_lanes = tmem + lanes + 32 * half;
        // writes part i of chunk u from registers, 16 columns at a time
        auto put_part = [&](int u, int i, int cols, const uint32_t(&out)[16]) {
            tmem_st_16x32(part_lanes + (static_cast<uint32_t>(16 * cols) << 16) + Turn::part(3 * u + i),
                          out);
        };
        auto part_done = [&](int u, int i) {
            tmem_wait_st();
            tc_fence_before();
            arrive(kPart + (3 * u + i) % Turn::kSlots);
        };
        auto part_free = [&](int u, int i) {
            const int j = 3 * u + i;
            return j < Turn::kSlots || wait_part(kPartFree, j - Turn::kSlots);
        };
        auto first_part = [&](int u) {
            const bool cut = it.rows - u * C < C;
            if (!(wait3(kFullV, u) && (!cut || wait2(kFull, u)) && wait2(kGFull, u) && part_free(u, 0)))
                return false;
            tc_fence_after();
            uint8_t *k_tile = sm + Smem::kK + (u & 1) * Smem::kTile;
            uint8_t *v_tile = sm + Smem::kV + u % 3 * Smem::kTile;
            if (cut) {
                // the next sequence's rows, which may hold anything: no part of any product
                // (each warp its own part of V, and as much of K)
                for (int i = lane; i < 256; i += 32) {
                    const int t = 64 * half + (i >> 2);
                    const uint32_t at = ((warp & 3) >> 1) * kBlk + at_tile(t, 4 * (warp & 1) + (i & 3));
                    if (u * C + t >= it.rows) {
                        *reinterpret_cast<uint4 *>(k_tile + at) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(v_tile + at) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            const Gates &g = gates[u & 1];
            decay = g.all;
            if (STATE) total += g.total;
            Pair w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 x =
                    *reinterpret_cast<const float2 *>(g.w + 64 * half + 8 * k + 2 * (lane & 3));
                w[k] = pair_of(x.x, x.y);
            }
            arrive(kGFree + (u & 1));
            // lanes 0-7 point at 8 tokens of 8 columns, 8-15 at the next columns', 16-31 at the
            // next tokens'
            const int q = warp & 3, t = 64 * half + (lane >> 4) * 8 + (lane & 7);
            const uint32_t from = smem_u32(v_tile) + (q >> 1) * kBlk + t * 128;
#pragma unroll
            for (int cols = 0; cols < 2; ++cols) {
                const int group = (4 * (q & 1) + 2 * cols + ((lane >> 3) & 1)) ^ (t & 7);
                uint32_t out[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t v[4];
                    load_transposed(from + k * 2048 + (group << 4), v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Pair x = mul2(w[2 * k + j / 2], widen(v[j]));
                        out[4 * k + j] = narrow(x);
                        left[cols][4 * k + j] = left_of(x, out[4 * k + j]);
                    }
                }
                put_part(u, 0, cols, out);
            }
            part_done(u, 0);
            return true;
        };
        auto next_part = [&](int u, int i) {
            if (!part_free(u, i)) return false;
            tc_fence_after();
#pragma unroll
            for (int cols = 0; cols < 2; ++cols) {
                uint32_t out[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    out[k] = narrow(left[cols][k]);
                    left[cols][k] = left_of(left[cols][k], out[k]);
                }
                put_part(u, i, cols, out);
            }
            part_done(u, i);
            return true;
        };
        if (STATE) {
            // h0 is kept for the second launch, whose blocks may write hT over it
            if (it.seg == 0 && p.h0) {
                add_state(p.h0 + state_at(it.n), 0.f);
                put_state(p.seg_state + state_at(it.slot + it.parts - 1));
                clear();
            }
        } else {
            if (p.h0)
                add_state(it.parts > 1 ? p.seg_state + state_at(it.slot + it.parts - 1)
                                       : p.h0 + state_at(it.n), 0.f);
            for (int m = 0; m < it.seg; ++m)
                add_state(p.seg_state + state_at(it.slot + m),
                          exp_centred(p.seg_log[static_cast<long long>(it.slot + m) * p.H + h]));
            if (nch > 0) put_copy();
        }
        bool ok = nch == 0 || first_part(0);
#pragma unroll 1
        for (int u = 0; ok && u < nch; ++u) {
            const Pair a = pair_of(decay, decay);
#pragma unroll 1
            for (int i = 1; ok && i < 3; ++i) ok = next_part(u, i);
            if (!ok || (u + 1 < nch && !(ok = first_part(u + 1)))) break;
            if (!(ok = wait2(kSum, u))) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                uint32_t x[32];
                tmem_ld32(tmem + lanes + Turn::sum(u) + 64 * half + i, x);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    S[(i + j) / 2] = fma2(a, S[(i + j) / 2], pair_of(x[j], x[j + 1]));
            }
            tc_fence_before();
            arrive(kSumFree + u % Turn::kSums);
            if (!STATE && u + 1 < nch) {
                if (!(ok = wait1(kQS, u))) break;
                put_copy();
            }
        }
        if (ok) {
            if (STATE) {
                put_state(p.seg_state + state_at(it.slot + it.seg));
                if (tid == 0 && tile == 0)
                    p.seg_log[static_cast<long long>(it.slot + it.seg) * p.H + h] = total;
            } else if (p.hT && it.seg == it.parts - 1) {
                put_state(p.hT + state_at(it.n));
            }
        }
    } else if (warp < 12) {
        // ================================================================ scores and outputs
        registers_down<112>();
        const int w = warp & 3, t = 32 * w + lane;
        const uint32_t at = tmem + lanes + kTScore;
        auto walk = [&](auto fine_scores) {
            constexpr bool FINE = decltype(fine_scores)::value;
#pragma unroll 1
            for (int u = 0; u < (FINE ? min(nch, 1) : nch); ++u) {
                if (!(wait2(kGFull, u) && wait1(kScore, u))) break;
                tc_fence_after();
                const Gates &g = gates[u & 1];
                const float4 *e4 = reinterpret_cast<const float4 *>(g.e);
                const bool deep = g.deep, steep = g.steep, plain = !deep && !FINE;
                const float own = g.e[t];
                // G_t - R_t, in two parts as -G_i; and what of it is added to each -G_i by itself
                const float base = deep ? -own - fmaxf(-own, kFloor) : 0.f, on = steep ? 0.f : base;
                const uint32_t two = steep ? g.rest[t / 2] : 0u;
                const float base_rest = -__uint_as_float(t & 1 ? two & 0xffff0000u : two << 16);
                const float f = p.scale * (deep ? ex2f(fmaxf(-own, kFloor)) : 1.f / own);
                // the tokens of warps before this one's, then its own, then those behind: 32 scores
                // become 16 columns, one block behind the other; or, in two parts, 32 in their place
#pragma unroll 1
                for (int b = 0; b <= w; ++b) {
                    uint32_t r[32], out[16];
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
                    if (steep) {
                        // the differences of the sums, then of their rests
                        const Pair sum = pair_of(base, base), rest = pair_of(base_rest, base_rest);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t *of = g.rest + 16 * b + 2 * j;
                            const float2 x = both(add2(add2(pair_of(e[j].x, e[j].y), sum),
                                                       add2(widen(of[0]), rest)));
                            const float2 y = both(add2(add2(pair_of(e[j].z, e[j].w), sum),
                                                       add2(widen(of[1]), rest)));
                            e[j] = make_float4(x.x, x.y, y.x, y.y);
                        }
                    }
                    if (plain) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 x = e[j / 4];
                            out[j / 2] = narrow(mul2(pair_of(r[j], r[j + 1]), pair_of(x.x, x.y)));
                            out[j / 2 + 1] = narrow(mul2(pair_of(r[j + 2], r[j + 3]), pair_of(x.z, x.w)));
                        }
                    } else {
                        uint32_t rest[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float f0 = j % 4 ? e[j / 4].z : e[j / 4].x;
                            float f1 = j % 4 ? e[j / 4].w : e[j / 4].y;
                            if (deep) {
                                // of a later token it may be infinite: a masked score stays 0
                                f0 = 32 * b + j <= t ? ex2f(on + f0) : 0.f;
                                f1 = 32 * b + j + 1 <= t ? ex2f(on + f1) : 0.f;
                            }
                            const Pair x = mul2(pair_of(r[j], r[j + 1]), pair_of(f0, f1));
                            out[j / 2] = narrow(x);
                            if (FINE) rest[j / 2] = narrow(left_of(x, out[j / 2]));
                        }
                        if (FINE) tmem_st16(at + 32 * b + 16, rest);
                    }
                    tmem_st16(at + (FINE ? 32 : 16) * b, out);
                }
                uint32_t none[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) none[j] = 0u;
#pragma unroll 1
                for (int b = w + 1; b < 4; ++b) {
                    tmem_st16(at + (FINE ? 32 : 16) * b, none);
                    if (FINE) tmem_st16(at + 32 * b + 16, none);
                }
                // q_t S of rows below the floor, in place before P V is added (8 prompts of 2,048 tokens, a
                // ninth of whose heads forget as fast, 59.5 us for 57.8 without)
                if (deep) {
                    if (!wait1(kQS, u)) break;
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, base < 0.f)) {
                        const float left = ex2f(base + base_rest);
#pragma unroll 1
                        for (int c = 0; c < 64 * cblocks; c += 32) {
                            uint32_t r[32], out[16];
                            tmem_ld32(tmem + lanes + kTOut + c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; j += 16) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    out[i] = __float_as_uint(left * __uint_as_float(r[j + i]));
                                tmem_st16(tmem + lanes + kTOut + c + j, out);
                            }
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(kP);
                arrive(kGFree + (u & 1));
                // the outputs of row t
                const Pair ff = pair_of(f, f);
                const int there = u * C + t < it.rows ? p.dv - c0 : 0;
                __nv_bfloat16 *to =
                    p.o + (static_cast<long long>(it.row + u * C + t) * p.H + h) * p.dv + c0;
                if (!wait2(kDone, u)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 64 * cblocks; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kTOut + c, r);
                    tmem_wait_ld();
                    if (c + 32 == 64 * cblocks) {
                        tc_fence_before();
                        arrive(kOFree);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[j] = narrow(mul2(ff, pair_of(r[i + 2 * j], r[i + 2 * j + 1])));
                        if (p.wide_store) {
                            if (c + i < there) store32(to + c + i, v);
                        } else {
                            if (c + i < there)
                                *reinterpret_cast<uint4 *>(to + c + i) =
                                    make_uint4(v[0], v[1], v[2], v[3]);
                            if (c + i + 8 < there)
                                *reinterpret_cast<uint4 *>(to + c + i + 8) =
                                    make_uint4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
            }
        };
        if (fine) walk(std::true_type{});
        else if (!STATE) walk(std::false_type{});
    } else if (warp == 12) {
        // ================================================================ loads
        registers_down<64>();
        int ks = 0, qs = 0, vs = 0;   // loads queued
        auto load_k = [&](int u) {
            uint64_t *full = &bar[kFull + (u & 1)];
            warp_expect_tx(full, kblocks * kBlk);
            for (int b = 0; b < kblocks; ++b)
                warp_tma_load_3d(sm + Smem::kK + (u & 1) * Smem::kTile + b * kBlk, &p.tk, full,
                                 b * 64, hk * p.k_step, it.row + u * C);
            ks = u + 1;
        };
        auto load_q = [&](int u) {
            if (STATE) return;
            warp_expect_tx(&bar[kFullQ], kblocks * kBlk);
            for (int b = 0; b < kblocks; ++b)
                warp_tma_load_3d(sm + Smem::kQ + b * kBlk, &p.tq, &bar[kFullQ], b * 64,
                                 hk * p.q_step, it.row + u * C);
            qs = u + 1;
        };
        auto load_v = [&](int u) {
            uint64_t *full = &bar[kFullV + u % 3];
            warp_expect_tx(full, cblocks * kBlk);
            for (int b = 0; b < cblocks; ++b)
                warp_tma_load_3d(sm + Smem::kV + u % 3 * Smem::kTile + b * kBlk, &p.tv, full,
                                 c0 + b * 64, h * p.v_step, it.row + u * C);
            vs = u + 1;
        };
        // the first chunks' tiles, then each as soon as the last product of the tile before it in
        // its place is done
        if (nch > 0) load_k(0), load_q(0), load_v(0);
        if (nch > 1) load_k(1), load_v(1);
        if (nch > 2) load_v(2);
#pragma unroll 1
        for (int u = 0; u + 1 < nch; ++u) {
            if (!STATE && !wait1(kQS, u)) break;
            load_q(u + 1);
            if (u + 2 < nch) {
                if (!wait2(kSum, u)) break;
                load_k(u + 2);
            }
            if (u + 3 < nch) {
                if (!STATE && !wait2(kDone, u)) break;
                load_v(u + 3);
            }
        }
        // loads that an expired wait left under way land before the block gives up its memory
        for (int u = max(0, ks - 2); u < ks; ++u) wait2(kFull, u);
        for (int u = max(0, vs - 3); u < vs; ++u) wait3(kFullV, u);
        if (qs > 0) wait1(kFullQ, qs - 1);
    } else if (warp == 13) {
        // ================================================================ gates
        registers_down<64>();
        float g[4], next[4];
        if (nch > 0) load_gates(p, it.row, min(C, it.rows), h, next);
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = next[j];
            if (u + 1 < nch)
                load_gates(p, it.row + (u + 1) * C, min(C, it.rows - (u + 1) * C), h, next);
            if (u >= 2 && !wait2(kGFree, u - 2)) break;
            write_gates<STATE>(g, gates[u & 1], fine);
            arrive(kGFull + (u & 1));
        }
    } else if (warp == 14) {
        // ================================================================ products
        registers_down<64>();
        // a step of 16 of the common dimension, in descriptors: 16 rows of a tile whose rows are
        // that dimension, 32 bytes of a row (and on to the next tile of 64 after four) otherwise
        constexpr uint64_t kRows = 2048 >> 4, kBytes32 = 32 >> 4, kNext = (kBlk - 96) >> 4;
        // [columns][tokens] by K [tokens][channels]; Q [t][c] by K [i][c]; by S [columns][c]; scores
        // by V [tokens][columns]
        const uint32_t id_sum = idesc_bf16(128, 64 * kblocks, false, true);
        const uint32_t id_score = idesc_bf16(C, C, false, false);
        const uint32_t id_qs = idesc_bf16(C, 64 * cblocks, false, false);
        const uint32_t id_pv = idesc_bf16(C, 64 * cblocks, false, true);
#pragma unroll 1
        for (int u = 0; u < nch; ++u) {
            const uint32_t k_tile = a0 + Smem::kK + (u & 1) * Smem::kTile;
            bool ok = wait2(kFull, u) && (u < Turn::kSums || wait_sum_free(u - Turn::kSums));
#pragma unroll 1
            for (int part = 0; ok && part < 3; ++part) {
                const int j = 3 * u + part;
                if (!(ok = wait_part(kPart, j))) break;
                tc_fence_after();
                uint64_t k = sw128_desc(k_tile, kBlk, 1024);
                uint32_t v = tmem + Turn::part(j);
#pragma unroll 1
                for (int i = 0; i < C / 16; ++i, k += kRows, v += 8)
                    warp_mma_bf16_ts(tmem + Turn::sum(u), v, k, id_sum, part + i > 0);
                warp_mma_commit(&bar[kPartFree + j % Turn::kSlots]);
                if (part > 0 || STATE) continue;
                // the scores of chunk u - 1 lay where these go
                if (!(ok = wait1(kFullQ, u) && (u == 0 || wait2(kDone, u - 1)))) break;
                tc_fence_after();
                uint64_t q = sw128_desc(a0 + Smem::kQ, 16, 1024);
                k = sw128_desc(k_tile, 16, 1024);
#pragma unroll 1
                for (int i = 0; i < ksteps; ++i) {
                    warp_mma_bf16_ss(tmem + kTScore, q, k, id_score, i > 0);
                    const uint64_t on = (i & 3) == 3 ? kNext : kBytes32;
                    q += on;
                    k += on;
                }
                warp_mma_commit(&bar[kScore]);
                if (!(ok = wait1(kCopy, u) && (u == 0 || wait1(kOFree, u - 1)))) break;
                tc_fence_after();
                q = sw128_desc(a0 + Smem::kQ, 16, 1024);
                k = sw128_desc(a0 + Smem::kS, 16, 1024);
#pragma unroll 1
                for (int i = 0; i < ksteps; ++i) {
                    warp_mma_bf16_ss(tmem + kTOut, q, k, id_qs, i > 0);
                    const uint64_t on = (i & 3) == 3 ? kNext : kBytes32;
                    q += on;
                    k += on;
                }
                warp_mma_commit(&bar[kQS]);
            }
            if (!ok) break;
            warp_mma_commit(&bar[kSum + (u & 1)]);
            if (STATE) continue;
            if (!wait1(kP, u)) break;
            tc_fence_after();
            uint64_t y = sw128_desc(a0 + Smem::kV + u % 3 * Smem::kTile, kBlk, 1024);
            if (!fine) {
#pragma unroll 1
                for (int i = 0; i < C / 16; ++i, y += kRows)
                    warp_mma_bf16_ts(tmem + kTOut, tmem + kTScore + 8 * i, y, id_pv, 1u);
            } else {
#pragma unroll 1
                for (int i = 0; i < C / 8; ++i) {
                    // both parts of 16 tokens' scores
                    const uint32_t score =
                        tmem + kTScore + (i >> 2) * 32 + (i & 1) * 16 + (i >> 1 & 1) * 8;
                    warp_mma_bf16_ts(tmem + kTOut, score, y + (i >> 1) * kRows, id_pv, 1u);
                }
            }
            warp_mma_commit(&bar[kDone + (u & 1)]);
        }
        // every product ends before TMEM and shared memory are given up
        warp_mma_commit(&bar[kDrain]);
        wait1(kDrain, 0);
    } else {
        registers_down<64>();
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

// How long a launch takes, in chunks: `items` segments (of at most `longest` chunks, `chunks` in all)
// for each of `lanes` heads and column tiles, longest first, on the SMs.  The less of whole rounds of
// the longest, and of everybody's share with half of the longest for an uneven end.  (Of blocks
// that are all alike somewhat more than a round is more than it says: 10 prompts of 16 chunks
// and 16 heads come to 28, where two rounds are 36.)
double launch_time(long long items, int longest, long long chunks, int lanes, double begin) {
    constexpr double kSms = 152;
    const double blocks = static_cast<double>(items) * lanes, most = longest + begin;
    if (blocks <= kSms) return most;
    return std::min(std::ceil(blocks / kSms) * most,
                    (chunks + items * begin) * lanes / kSms + 0.5 * most);
}

// Cutting costs a launch that walks all but the last segments for their sums (kSumCost of a chunk's
// whole work each), and each block what it takes to begin (kItem) and to read the states before it
// (kJoin each), all in chunks.  Of no cut and of 2 to 32 parts for the longest sequence, the one
// that launch_time says is the quickest.  Two sequences of 32,768 tokens, 16 heads of 128 and 256:
// 7 parts 559 us, 732 in one, 587, 605 and 602 in 2, 4 and 9.
Plan make_plan(const int *cu, int N, int H, int dv) {
    constexpr double kSumCost = 0.5, kBegin = 1, kItem = 2, kJoin = 0.2;
    const int lanes = H * ((dv + kCols - 1) / kCols);
    int longest = 0;
    long long all = 0;
    for (int n = 0; n < N; ++n) {
        longest = std::max(longest, chunks_of(cu, n));
        all += chunks_of(cu, n);
    }
    Plan best = {INT_MAX, 0};
    double least = launch_time(N, longest, all, lanes, kItem);
    for (int k = 2; k <= 32 && k <= longest; ++k) {
        const int most = (longest + k - 1) / k;
        // not even with the first launch for nothing
        if (std::max<double>(most, all * lanes / 152.) + kBegin >= least) continue;
        long long items = 0, first_items = 0, first = 0, slots = 0;
        for (int n = 0; n < N; ++n) {
            const int c = chunks_of(cu, n), parts = parts_of(c, most);
            items += parts;
            if (parts == 1) continue;
            first_items += parts - 1;
            first += c - c / parts;
            slots += parts;
        }
        const double cost = launch_time(items, most, all, lanes, kItem + kJoin * (k - 1)) + kBegin +
                            kSumCost * launch_time(first_items, most, first, lanes, kItem);
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
    const Span work = span_of(scratch, need, 1);
    if (meets_any(work, in) || meet(work, out) || meet(work, begin) || meet(work, end))
        return GLA_ERR_ARG;
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
