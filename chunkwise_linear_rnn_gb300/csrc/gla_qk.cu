// gla_qk.cu — norms of the query and key rows with the rotation by position, in
// one pass from the token-major layout to the head-first one:
//     y = R_p(w * x * r),   r = 1 / sqrt(sum_i x_i^2 / n + eps),
// and its backward: with z = R_p^T dy, g = w * z and unit = x r,
//     dw = sum over rows of z * unit,   dx = r (g - unit * <g, unit> / n).
//
// A warp takes one token and walks its heads, a group of lanes (8 values to a lane) for
// each row: the cosines and sines of the token stay in registers for all its heads.
// Eight warps take eight neighbouring tokens, so that the head-first stores of a block are
// contiguous runs of eight rows.
//
// Bound by HBM (4 bytes a bf16 value forward, 6 backward) where instructions leave it room:
// about 90 a round of 8 values a lane forward, 200 backward.  Measured on one GB300, bf16:
// B2 T32768, 16+16 heads of 128, no rotation 164 us (6.6 TB/s of a copy's 6.67); B8 T2048,
// 16+16 heads of 128, rotated 46 us (5.8 TB/s); B4 T4096, 32+8 heads of 64, half of each
// rotated, 34 us (4.9 TB/s) and backward 54 us (4.7 TB/s) with its second launch.
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

// Thread blocks of the backward, at most: 2 for each of 152 SMs.  A constant, since the scratch
// that they leave their sums in is sized by d alone.
constexpr int kPartials = 304;
constexpr long long kFwdBlocks = 8;   // thread blocks of the forward for each SM, at most

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
    int chunk;               // heads (q's, then k's) of a block
    long long first, end;    // backward: the launch's tokens
    float inv_n, eps;
};

// Where the backward's weight gradients go, and their sums over several launches.
struct WeightGrads {
    float *q, *k;
    double *so_far;          // [2][d]
};

constexpr int kWarps = 8;

// ---------------------------------------------------------------- values and pairs

// Two fp32 values, for operations on both in one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float a, float b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
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
__device__ __forceinline__ Pair swapped(Pair a) {
    const float2 v = both(a);
    return pair_of(v.y, v.x);
}

// A lane's 8 values of a row: blocks A and B of 4.  With halves, A lies in the first half of
// the rotated part and B at the same place of the second; elsewhere B follows A.
template <typename E>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int ia, int ib) {
        a = *reinterpret_cast<const uint2 *>(p + ia);
        b = *reinterpret_cast<const uint2 *>(p + ib);
    }
    __device__ __forceinline__ void load_two(const void *pa, const void *pb) {
        a = *static_cast<const uint2 *>(pa);
        b = *static_cast<const uint2 *>(pb);
    }
    __device__ __forceinline__ static Pair widen(unsigned w) {
        return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ void get(Pair (&v)[4]) const {
        v[0] = widen(a.x), v[1] = widen(a.y), v[2] = widen(b.x), v[3] = widen(b.y);
    }
    __device__ __forceinline__ static unsigned narrow(Pair p) {
        const float2 v = both(p);
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const unsigned *>(&h);
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, int ia, int ib,
                                                 const Pair (&v)[4]) {
        *reinterpret_cast<uint2 *>(p + ia) = make_uint2(narrow(v[0]), narrow(v[1]));
        *reinterpret_cast<uint2 *>(p + ib) = make_uint2(narrow(v[2]), narrow(v[3]));
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, int ia, int ib) {
        a = *reinterpret_cast<const float4 *>(p + ia);
        b = *reinterpret_cast<const float4 *>(p + ib);
    }
    __device__ __forceinline__ void load_two(const void *pa, const void *pb) {
        a = *static_cast<const float4 *>(pa);
        b = *static_cast<const float4 *>(pb);
    }
    __device__ __forceinline__ void get(Pair (&v)[4]) const {
        v[0] = pair_of(a.x, a.y), v[1] = pair_of(a.z, a.w);
        v[2] = pair_of(b.x, b.y), v[3] = pair_of(b.z, b.w);
    }
    __device__ __forceinline__ static void store(float *p, int ia, int ib, const Pair (&v)[4]) {
        const float2 x = both(v[0]), y = both(v[1]), z = both(v[2]), w = both(v[3]);
        *reinterpret_cast<float4 *>(p + ia) = make_float4(x.x, x.y, y.x, y.y);
        *reinterpret_cast<float4 *>(p + ib) = make_float4(z.x, z.y, w.x, w.y);
    }
};

// The sum over the lanes of a group.
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ float total(const Pair (&v)[4], const Pair (&w)[4]) {
    const float2 s = both(fma2(v[3], w[3], fma2(v[2], w[2], fma2(v[1], w[1], mul2(v[0], w[0])))));
    return s.x + s.y;
}

// ---------------------------------------------------------------- angles

// A frequency as 2^64ths of a turn per position, without its whole turns: the angle of any
// whole position is then a product modulo 2^64.  The frequency's 53-bit significand times
// 2^64 / (2 pi), shifted by its exponent, all in integers: off by 2^-64 of a turn for
// frequencies up to 1, with none of the few fp64 units in it.
__device__ __forceinline__ unsigned long long turn_of(double inv_freq) {
    const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(inv_freq));
    const int e = static_cast<int>((bits >> 52) & 0x7ff) - 1023;
    const unsigned long long m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
    const unsigned long long c = 0x28be60db9391054aull;   // 2^64 / (2 pi)
    const unsigned long long lo = m * c, hi = __umul64hi(m, c);
    const int s = 52 - e;
    unsigned long long t;
    if (s >= 128) t = 0;
    else if (s >= 64) t = hi >> (s - 64);
    else if (s > 0) t = (hi << (64 - s)) | (lo >> s);
    else t = s > -64 ? lo << -s : 0;
    return bits >> 63 ? 0 - t : t;
}

// cos and sin of a phase in 2^32nds of a turn (a third of the instructions of sincospif,
// which does not know that its argument is reduced): the nearest quarter by integers, then
// Chebyshev fits in the square of what is left, |x| <= 1/2 quarters (sin = x S(x^2), cos =
// 1 + x^2 C(x^2)).  The fits are within a rounding of 2^-24; with those of x, its square and
// the products the values are off by 1.72 * 2^-24 at most and 0.35 * 2^-24 in the root mean
// square (33 million phases; a rounded 64-bit value: 0.5 and 0.24).
__device__ __forceinline__ float2 cos_sin(unsigned phase) {
    const unsigned quarter = (phase + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int>(phase - (quarter << 30))) * 9.313225746154785e-10f;
    const float z = x * x;
    const float s = x * fmaf(fmaf(fmaf(-4.6021174639463425e-3f, z, 7.968020439147949e-2f), z,
                                  -0.6459634900093079f), z, 1.5707963705062866f);
    const float c = fmaf(fmaf(fmaf(fmaf(9.06734901946038e-4f, z, -2.086152695119381e-2f), z,
                                   0.253669410943985f), z, -1.2337005138397217f), z, 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2(__uint_as_float(__float_as_uint(a) ^ ((quarter + 1) << 30 & 0x80000000u)),
                       __uint_as_float(__float_as_uint(b) ^ (quarter << 30 & 0x80000000u)));
}

// A lane's part of every row: its values, and the angles that it works out for itself and the
// same lanes of the warp's other groups.
template <int LANES, bool HALVES>
struct Lane {
    static constexpr int kRows = 32 / LANES, kOwn = 4 / kRows;   // groups; angles of each
    int ia, ib;              // its blocks of 4 values
    bool there, turns;       // it has values; they are rotated
    unsigned long long turn[kOwn];

    __device__ __forceinline__ Lane(const QkArgs &p, int lane) {
        const int j = lane % LANES;
        there = 8 * j < p.d;
        turns = 8 * j < p.rot;
        ia = 8 * j;
        ib = ia + 4;
        if (HALVES && turns) ia = 4 * j, ib = 4 * j + p.rot / 2;
        if (!there) ia = 0, ib = 4;   // reads what another lane reads, writes nothing
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            turn[i] = turns ? turn_of(p.inv_freq[4 * j + lane / LANES * kOwn + i]) : 0;
    }
};

// The cosines and sines of a token: c, s of the lane's pairs, two by two for halves (with -s in
// m), each twice for neighbours (u, v) -> (u, v) c + (v, u) (-s, s) (with (s, -s) in m).
template <int LANES, bool HALVES>
struct Angles {
    Pair c[HALVES ? 2 : 4], s[HALVES ? 2 : 4], m[HALVES ? 2 : 4];

    __device__ __forceinline__ void at(const Lane<LANES, HALVES> &l, long long pos) {
        using L = Lane<LANES, HALVES>;
        float2 own[L::kOwn], v[4];
#pragma unroll
        for (int i = 0; i < L::kOwn; ++i)
            own[i] = cos_sin(static_cast<unsigned>(
                (l.turn[i] * static_cast<unsigned long long>(pos)) >> 32));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = own[i % L::kOwn];
            if constexpr (L::kRows > 1) {
                const int from = i / L::kOwn * LANES + (threadIdx.x & (LANES - 1));
                v[i].x = __shfl_sync(0xffffffffu, v[i].x, from);
                v[i].y = __shfl_sync(0xffffffffu, v[i].y, from);
            }
        }
#pragma unroll
        for (int i = 0; i < (HALVES ? 2 : 4); ++i) {
            const float2 a = HALVES ? v[2 * i] : v[i], b = HALVES ? v[2 * i + 1] : v[i];
            c[i] = pair_of(a.x, b.x);
            s[i] = pair_of(HALVES ? a.y : -a.y, b.y);
            m[i] = pair_of(HALVES ? -a.y : a.y, -b.y);
        }
    }
    // Turns the four pairs by their angles, or back.
    template <bool BACK>
    __device__ __forceinline__ void turn(Pair (&v)[4]) const {
        if constexpr (HALVES) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Pair u = v[i], w = v[i + 2];
                v[i] = fma2(w, BACK ? s[i] : m[i], mul2(u, c[i]));
                v[i + 2] = fma2(u, BACK ? m[i] : s[i], mul2(w, c[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = fma2(swapped(v[i]), BACK ? m[i] : s[i], mul2(v[i], c[i]));
        }
    }
};

// ---------------------------------------------------------------- the kernels

// Loads the lane's weights (1 without a weight).
__device__ __forceinline__ void weights(const float *w, int ia, int ib, Pair (&v)[4]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pair_of(1.f, 1.f);
        return;
    }
    Eight<float> e;
    e.load(w, ia, ib);
    e.get(v);
}

// Heads [from, to) of q (which = 0) or k of those that the block takes.
struct Heads {
    int from, to;
};
__device__ __forceinline__ Heads heads_of(const QkArgs &p, int which) {
    const int a = blockIdx.y * p.chunk - (which ? p.H[0] : 0);
    return {max(a, 0), min(a + p.chunk, p.H[which])};
}

// n / T, in 32 bits where they are enough.
__device__ __forceinline__ int batch_of(const QkArgs &p, long long n, long long tokens) {
    return tokens >> 32 ? static_cast<int>(n / p.T)
                        : static_cast<int>(static_cast<unsigned>(n) / static_cast<unsigned>(p.T));
}

// PART: only the first rot < d values are rotated, so that some lanes rotate and some do not.
template <typename E, int LANES, bool HALVES, bool PART>
__global__ void __launch_bounds__(32 * kWarps, 4) qk_fwd_kernel(const __grid_constant__ QkArgs p) {
    constexpr int ROWS = 32 / LANES, AHEAD = 4;   // rows of a warp at once, and loads ahead
    const int lane = threadIdx.x & 31, row = lane / LANES;
    const Lane<LANES, HALVES> l(p, lane);
    const long long tokens = static_cast<long long>(p.B) * p.T;
    for (long long n = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5); n < tokens;
         n += static_cast<long long>(gridDim.x) * kWarps) {
        const int b = batch_of(p, n, tokens), t = static_cast<int>(n - static_cast<long long>(b) * p.T);
        Angles<LANES, HALVES> turn;
        if (p.rot) turn.at(l, p.pos ? p.pos[b * p.lay.pos_sb + t] : t);
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const Heads hs = heads_of(p, which);
            if (hs.from >= hs.to) continue;
            const long long sh = which ? p.lay.k_sh : p.lay.q_sh;
            const E *x = static_cast<const E *>(p.x[which]) +
                         (which ? b * p.lay.k_sb + t * p.lay.k_st : b * p.lay.q_sb + t * p.lay.q_st);
            const size_t out_h = static_cast<size_t>(p.T) * p.d;
            E *y = static_cast<E *>(p.y[which]) + static_cast<size_t>(b) * p.H[which] * out_h +
                   static_cast<size_t>(t) * p.d;
            Pair w[4];
            weights(p.w[which], l.ia, l.ib, w);
            const auto finish = [&](const Eight<E> &raw, E *to, bool mine) {
                Pair v[4];
                raw.get(v);
                const float sum = group_sum<LANES>(l.there ? total(v, v) : 0.f);
                const float r = rsqrtf(fmaf(sum, p.inv_n, p.eps));
                const Pair rr = pair_of(r, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = mul2(mul2(v[k], rr), w[k]);
                if (PART ? l.turns : p.rot > 0) turn.template turn<false>(v);
                if (mine) Eight<E>::store(to, l.ia, l.ib, v);
            };
            int h = hs.from;
#pragma unroll 1
            for (; h + ROWS * AHEAD <= hs.to; h += ROWS * AHEAD) {
                Eight<E> raw[AHEAD];
                const E *from = x + (h + row) * sh;
                E *to = y + (h + row) * out_h;
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    raw[i].load(from, l.ia, l.ib);
                    from += ROWS * sh;
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    finish(raw[i], to, l.there);
                    to += ROWS * out_h;
                }
            }
            // the last heads, a round at a time; lanes past the end take the last head again
#pragma unroll 1
            for (; h < hs.to; h += ROWS) {
                Eight<E> raw;
                raw.load(x + min(h + row, hs.to - 1) * sh, l.ia, l.ib);
                finish(raw, y + (h + row) * out_h, l.there && h + row < hs.to);
            }
        }
    }
}

// Values copied to shared memory in the background.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// The rounds of a warp, one after another: a token's heads of q, then of k, then the next
// token.  x and dy point at this lane's row.
template <typename E, int ROWS>
struct Rounds {
    long long n;             // token
    int h, to;               // head of the round, and the part's end
    bool of_k;
    const E *x, *dy;
    long long step, dy_step;

    __device__ __forceinline__ void begin(const QkArgs &p, long long token, long long tokens,
                                          int row) {
        n = token;
        const Heads q = heads_of(p, 0);
        part(p, q.from >= q.to, tokens, row);
    }
    __device__ __forceinline__ void part(const QkArgs &p, bool k, long long tokens, int row) {
        of_k = k;
        if (n >= tokens) return;
        const Heads hs = heads_of(p, k);
        h = hs.from;
        to = hs.to;
        const int b = batch_of(p, n, tokens);
        const long long t = n - static_cast<long long>(b) * p.T;
        const long long sh = k ? p.lay.k_sh : p.lay.q_sh;
        const long long out_h = static_cast<long long>(p.T) * p.d;
        x = static_cast<const E *>(k ? p.x[1] : p.x[0]) + (h + row) * sh +
            (k ? b * p.lay.k_sb + t * p.lay.k_st : b * p.lay.q_sb + t * p.lay.q_st);
        dy = static_cast<const E *>(k ? p.dy[1] : p.dy[0]) +
             (static_cast<long long>(b) * (k ? p.H[1] : p.H[0]) + h + row) * out_h + t * p.d;
        step = ROWS * sh;
        dy_step = ROWS * out_h;
    }
    __device__ __forceinline__ void next(const QkArgs &p, long long tokens, int row) {
        h += ROWS;
        x += step;
        dy += dy_step;
        if (h < to) return;
        const Heads k = heads_of(p, 1);
        if (!of_k && k.from < k.to) part(p, true, tokens, row);
        else begin(p, n + static_cast<long long>(gridDim.x) * kWarps, tokens, row);
    }
};

// Backward.  A queue of DEPTH rounds of x and dy for each warp is on its way to shared
// memory: each lane copies and reads its own values, so that no barrier stands between.
// (The same rows loaded two rounds ahead to registers: 70 us where this takes 54.)
template <typename E, int LANES, bool HALVES, bool PART>
__global__ void __launch_bounds__(32 * kWarps, 2)
    qk_bwd_kernel(const __grid_constant__ QkArgs p) {
    constexpr int ROWS = 32 / LANES, DEPTH = sizeof(E) == 2 ? 4 : 3;
    constexpr int PIECE = 4 * sizeof(E), PIECES = 4;   // a lane's blocks A and B of x and of dy
    __shared__ __align__(16) unsigned char s_queue[kWarps][DEPTH][PIECES][32][PIECE];
    static_assert(sizeof(s_queue) >= sizeof(float) * kWarps * ROWS * 8 * LANES, "the sums' space");
    const int lane = threadIdx.x & 31, row = lane / LANES;
    const Lane<LANES, HALVES> l(p, lane);
    const long long tokens = p.end;
    const long long start =
        p.first + blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5);
    auto *queue = s_queue[threadIdx.x >> 5];

    Rounds<E, ROWS> ask;
    ask.begin(p, start, tokens, row);
    const auto request = [&](int slot) {
        if (ask.n < tokens) {
            if (ask.h + row < ask.to) {   // the others' values go nowhere
                const uint32_t to = smem_u32(&queue[slot][0][lane][0]);
                copy_async<PIECE>(to, ask.x + l.ia);
                copy_async<PIECE>(to + 32 * PIECE, ask.x + l.ib);
                copy_async<PIECE>(to + 64 * PIECE, ask.dy + l.ia);
                copy_async<PIECE>(to + 96 * PIECE, ask.dy + l.ib);
            }
            ask.next(p, tokens, row);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) request(i);

    Pair dw[2][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[0][k] = dw[1][k] = pair_of(0.f, 0.f);
    int slot = 0;
    for (long long n = start; n < tokens; n += static_cast<long long>(gridDim.x) * kWarps) {
        Angles<LANES, HALVES> turn;
        if (p.rot) {
            const int b = batch_of(p, n, tokens);
            const long long t = n - static_cast<long long>(b) * p.T;
            turn.at(l, p.pos ? p.pos[b * p.lay.pos_sb + t] : t);
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const Heads hs = heads_of(p, which);
            if (hs.from >= hs.to) continue;
            E *dx = static_cast<E *>(p.y[which]) + (n * p.H[which] + hs.from + row) * p.d;
            Pair w[4];
            weights(p.w[which], l.ia, l.ib, w);
#pragma unroll 1
            for (int h = hs.from; h < hs.to; h += ROWS) {
                asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
                Pair v[4], z[4], g[4];
                Eight<E> raw;
                raw.load_two(&queue[slot][0][lane][0], &queue[slot][1][lane][0]);
                raw.get(v);
                raw.load_two(&queue[slot][2][lane][0], &queue[slot][3][lane][0]);
                raw.get(z);
                request(slot);
                slot = slot == DEPTH - 1 ? 0 : slot + 1;
                const bool mine = l.there && h + row < hs.to;
                if (PART ? l.turns : p.rot > 0) turn.template turn<true>(z);
#pragma unroll
                for (int k = 0; k < 4; ++k) g[k] = mul2(z[k], w[k]);
                const float sum = group_sum<LANES>(l.there ? total(v, v) : 0.f);
                const float dot = group_sum<LANES>(l.there ? total(g, v) : 0.f);
                const float r = rsqrtf(fmaf(sum, p.inv_n, p.eps));
                const float along = -(dot * r) * p.inv_n;   // - <g, unit> / n
                const Pair rr = pair_of(r, r), aa = pair_of(along, along);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const Pair unit = mul2(v[k], rr);
                    if (mine) dw[which][k] = fma2(z[k], unit, dw[which][k]);
                    v[k] = mul2(fma2(unit, aa, g[k]), rr);
                }
                if (mine) Eight<E>::store(dx, l.ia, l.ib, v);
                dx += ROWS * p.d;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    auto *s_dw = reinterpret_cast<float(*)[8 * LANES]>(&s_queue[0][0][0][0][0]);
    if (!p.partial) return;
    // the block's sums: the warps' and groups' one after another, q then k
    const size_t block = static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (l.there)
            Eight<float>::store(s_dw[(threadIdx.x >> 5) * ROWS + row], l.ia, l.ib, dw[which]);
        __syncthreads();
        for (int i = threadIdx.x; i < p.d; i += 32 * kWarps) {
            float v = 0.f;
#pragma unroll 8
            for (int k = 0; k < kWarps * ROWS; ++k) v += s_dw[k][i];
            p.partial[(block * 2 + which) * p.d + i] = v;
        }
    }
}

// The blocks' partial weight gradients, added in order in fp64.  Of several launches (`so_far`
// given) each adds its own to the sums of those before it; the last one writes the gradients.
__global__ void __launch_bounds__(1024)
    qk_weight_grad_kernel(const float *partial, int blocks, int d, float *gq, float *gk,
                          double *so_far, bool first, bool last) {
    __shared__ double s_sum[32][17];
    const int c = threadIdx.x & 15, part = threadIdx.x >> 4;   // 16 columns, 64 parts
    const int i = blockIdx.x * 16 + c;
    double v = 0.0;
#pragma unroll 4
    for (int b = part; b < blocks; b += 64) v += partial[static_cast<size_t>(b) * 2 * d + i];
    if (part >= 32) s_sum[part - 32][c] = v;
    __syncthreads();
    if (part < 32) s_sum[part][c] += v;
    __syncthreads();
    if (part != 0) return;
    v = 0.0;
    for (int k = 0; k < 32; ++k) v += s_sum[k][c];
    if (so_far) {
        if (!first) v += so_far[i];
        so_far[i] = v;
    }
    if (!last) return;
    float *g = i < d ? gq : gk;
    if (g) g[i < d ? i : i - d] = static_cast<float>(v);
}

// The work of a call as a grid: eight tokens to a block, and the heads in as many chunks
// (of whole rounds of the warps' rows) as fill the device with small batches.  `most`:
// blocks at most, the rest of the tokens taken by the same blocks.  `rounds_each`: rounds of a
// token that a block takes at most, as long as `most` blocks are enough for that.
dim3 grid_of(QkArgs &a, int rows, long long most, int rounds_each, int sms) {
    const long long tokens = static_cast<long long>(a.B) * a.T;
    const long long groups = (tokens + kWarps - 1) / kWarps;
    const int heads = a.H[0] + a.H[1], rounds = (heads + rows - 1) / rows;
    const long long want = std::max<long long>((4LL * sms + groups - 1) / groups,
                                               (rounds - 1) / rounds_each + 1);
    const int chunks = static_cast<int>(std::min<long long>({want, rounds, 65535, most}));
    a.chunk = (rounds + chunks - 1) / chunks * rows;
    const int y = (heads + a.chunk - 1) / a.chunk;
    return dim3(static_cast<unsigned>(std::max<long long>(1, std::min(groups, most / y))), y);
}

// Rows that a lane adds one after another in 32 bits for the weight gradients, at most: a
// token's many heads go to several blocks (enough for 300,000 heads; more add more), and a
// longer batch takes several launches, whose sums are added in 64 bits.  (As a test in the
// kernel, once a token, it took 5% of the time: 54 us -> 56.5 for B4 T4096, 32+8 heads of 64.)
constexpr int kSumRows = 1024;

template <typename E, int LANES, bool HALVES, bool PART>
int launch_bwd(QkArgs &a, const WeightGrads &to, int sms, cudaStream_t stream) {
    constexpr int ROWS = 32 / LANES;
    // q's and k's heads of a block may each end in a short round
    const dim3 grid = grid_of(a, ROWS, kPartials, a.partial ? kSumRows - 1 : INT_MAX, sms);
    const long long tokens = static_cast<long long>(a.B) * a.T;
    const long long each = std::max(1, kSumRows / (a.chunk / ROWS + 1));
    const long long step = a.partial ? each * grid.x * kWarps : tokens;
    for (a.first = 0; a.first < tokens; a.first = a.end) {
        a.end = std::min(a.first + step, tokens);
        qk_bwd_kernel<E, LANES, HALVES, PART><<<grid, 32 * kWarps, 0, stream>>>(a);
        if (a.partial)
            qk_weight_grad_kernel<<<2 * a.d / 16, 1024, 0, stream>>>(
                a.partial, grid.x * grid.y, a.d, to.q, to.k, step < tokens ? to.so_far : nullptr,
                a.first == 0, a.end == tokens);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    return 0;
}

template <typename E, int LANES, bool HALVES, bool PART, bool BACKWARD>
int launch_one(QkArgs &a, const WeightGrads &to, int sms, cudaStream_t stream) {
    if constexpr (BACKWARD) {
        return launch_bwd<E, LANES, HALVES, PART>(a, to, sms, stream);
    } else {
        const dim3 grid = grid_of(a, 32 / LANES, kFwdBlocks * sms, INT_MAX, sms);
        qk_fwd_kernel<E, LANES, HALVES, PART><<<grid, 32 * kWarps, 0, stream>>>(a);
        return static_cast<int>(cudaGetLastError());
    }
}

template <typename E, int LANES, bool BACKWARD>
int launch_lanes(QkArgs &a, const WeightGrads &to, int sms, cudaStream_t stream) {
    const bool halves = !a.interleaved, part = a.rot > 0 && a.rot < a.d;
    if (halves) return part ? launch_one<E, LANES, true, true, BACKWARD>(a, to, sms, stream)
                            : launch_one<E, LANES, true, false, BACKWARD>(a, to, sms, stream);
    return part ? launch_one<E, LANES, false, true, BACKWARD>(a, to, sms, stream)
                : launch_one<E, LANES, false, false, BACKWARD>(a, to, sms, stream);
}

template <typename E, bool BACKWARD>
int launch(QkArgs &a, const WeightGrads &to, int sms, cudaStream_t stream) {
    if (a.d <= 64) return launch_lanes<E, 8, BACKWARD>(a, to, sms, stream);
    if (a.d <= 128) return launch_lanes<E, 16, BACKWARD>(a, to, sms, stream);
    return launch_lanes<E, 32, BACKWARD>(a, to, sms, stream);
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
    // heads are counted on past the last in whole rounds of whole chunks
    if (static_cast<long long>(a.H[0]) + a.H[1] > 1LL << 30) return GLA_ERR_ARG;
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
    const int e = options->dtype == GLA_BF16 ? launch<__nv_bfloat16, false>(a, {}, sms, stream)
                                             : launch<float, false>(a, {}, sms, stream);
    return e == 0 ? GLA_OK : GLA_ERR_LAUNCH;
}

unsigned long gla_qk_norm_rope_bwd_scratch(int d) {
    return d > 0 ? 2ul * d * (gla::kPartials * sizeof(float) + sizeof(double)) : 0;
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
    WeightGrads to = {};
    if (grad_wq || grad_wk) {
        if (!scratch || !aligned(scratch, 16)) return GLA_ERR_ARG;
        if (scratch_bytes < gla_qk_norm_rope_bwd_scratch(d)) return GLA_ERR_SCRATCH;
        if (!aligned(grad_wq, 4) || !aligned(grad_wk, 4)) return GLA_ERR_ARG;
        a.partial = static_cast<float *>(scratch);
        to = {grad_wq, grad_wk, reinterpret_cast<double *>(a.partial + size_t{kPartials} * 2 * d)};
    }
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const int e = options->dtype == GLA_BF16 ? launch<__nv_bfloat16, true>(a, to, sms, stream)
                                             : launch<float, true>(a, to, sms, stream);
    return e == 0 ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // extern "C"
