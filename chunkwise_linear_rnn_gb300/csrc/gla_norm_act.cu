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
// block are then contiguous runs too.  The next token's rows are loaded while one is worked on
// (two ahead are slower: 255 us for 250 of B2 T32768, 16 heads of 256), and the offsets go on
// by additions (a division by T for each row took 40 us where it is 35 at B8 T2048).
//
// Bound by HBM where instructions leave it room (6 bytes a bf16 value forward with a gate, 10
// backward).  Measured on one GB300, bf16, gate: B2 T32768, 16 heads of 256, mean, weights and
// biases of every channel 252 us (6.4 TB/s of a copy's 6.79); B8 T2048, 16 heads of 128,
// head-first in, gate in a wider tensor 35.5 us (5.7 TB/s); B4 T4096 of the same forward 36 us and
// backward 70 us (4.8 TB/s) with its second launch, in fp32 62 us (6.5 TB/s) and 130 us (5.2 TB/s).
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
// Thread blocks of an SM that run at once, and of a launch (a second round of blocks only costs
// its beginning: twice as many forward 41.0 us for 40.4 at B8 T2048, 16 heads of 128, backward
// 134 for 123).  The backward's are a constant of 152 SMs, since its scratch is sized by the
// tensors alone.
template <typename E, int NB>
constexpr int kFwdPerSm = NB > 1 ? 2 : sizeof(E) == 2 ? 4 : 3;
constexpr long long kBwdBlocks = 304;    // 2 an SM, more where that keeps kSumRows
constexpr int kSumRows = 1024;           // rows that a lane adds in 32 bits

struct NormArgs {
    const void *x, *gate, *dy;
    const float *w, *b;
    void *y, *dx, *dgate;
    double *partial;         // backward with weights: see reduce_kernel
    gla_norm_act_layout lay;
    unsigned tokens, T;      // T = tokens where one stride steps over batch and tokens
    int H, d, groups;        // groups of the heads that a warp takes together
    int layer, silu, per_channel;
    float inv_d, eps;
};

// Two fp32 values, for operations on both in one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float a, float b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ Pair twice(float a) { return pair_of(a, a); }
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

// Eight neighbouring values of a row, as they lie in memory.
template <typename E>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        v = __ldg(reinterpret_cast<const uint4 *>(p));
    }
    __device__ __forceinline__ static Pair widen(unsigned w) {
        return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ void get(Pair (&x)[4]) const {
        x[0] = widen(v.x), x[1] = widen(v.y), x[2] = widen(v.z), x[3] = widen(v.w);
    }
    __device__ __forceinline__ static unsigned narrow(Pair p) {
        const float2 f = both(p);
        return pack_bf16x2(f.x, f.y);
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const Pair (&x)[4]) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(Pair (&x)[4]) const {
        x[0] = pair_of(a.x, a.y), x[1] = pair_of(a.z, a.w);
        x[2] = pair_of(b.x, b.y), x[3] = pair_of(b.z, b.w);
    }
    __device__ __forceinline__ static void store(float *p, const Pair (&x)[4]) {
        const float2 u = both(x[0]), v = both(x[1]), w = both(x[2]), z = both(x[3]);
        reinterpret_cast<float4 *>(p)[0] = make_float4(u.x, u.y, v.x, v.y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(w.x, w.y, z.x, z.y);
    }
};

template <int LANES>
__device__ __forceinline__ float group_sum(Pair v) {
    const float2 f = both(v);
    float s = f.x + f.y;
#pragma unroll
    for (int off = LANES / 2; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

// s(z) = 1 / (1 + exp(-z)).  Rows that end in bf16 take the hardware's 2^x and reciprocal (each
// within a few roundings of 2^-23), fp32 rows CUDA's own.
__device__ __forceinline__ Pair sigmoid(Pair z, __nv_bfloat16) {
    const float2 x = both(mul2(z, twice(-1.4426950408889634f)));
    const float2 d = both(add2(pair_of(ex2f(x.x), ex2f(x.y)), twice(1.f)));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    return pair_of(r.x, r.y);
}
__device__ __forceinline__ Pair sigmoid(Pair z, float) {
    const float2 x = both(z);
    return pair_of(1.f / (1.f + expf(-x.x)), 1.f / (1.f + expf(-x.y)));
}

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
                                             Pair (&w)[NB][4], Pair (&b)[NB][4]) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][e] = twice(1.f), b[i][e] = 0;
        if (!at.there[i]) continue;
        const int o = (p.per_channel ? at.h * p.d : 0) + at.c[i];
        Raw<float> r;
        if (p.w) r.load(p.w + o), r.get(w[i]);
        if (p.b) r.load(p.b + o), r.get(b[i]);
    }
}

// A walk over tokens n, n + step, ...: the offset of a row's start (in elements) goes on by what a
// step adds in whole sequences and tokens, and once more by what a token past a sequence's end is
// off, without a division after the first.
struct Walk {
    long long at, on, wrap;

    __device__ __forceinline__ Walk(const NormArgs &p, unsigned n, unsigned step, int h,
                                    long long sb, long long st, long long sh) {
        const unsigned b = n / p.T, q = step / p.T;
        at = b * sb + (n - b * p.T) * st + h * sh;
        on = q * sb + (step - q * p.T) * st;
        wrap = sb - p.T * st;
    }
    __device__ __forceinline__ void next(bool wraps) { at += wraps ? on + wrap : on; }
};
// The token of a walk: whether its step goes past the end of its sequence.
struct Token {
    unsigned n, t, step, rest;

    __device__ __forceinline__ Token(const NormArgs &p, unsigned first, unsigned by)
        : n(first), t(first % p.T), step(by), rest(by % p.T) {}
    __device__ __forceinline__ bool next(const NormArgs &p) {
        n += step;
        t += rest;
        const bool wraps = t >= p.T;
        if (wraps) t -= p.T;
        return wraps;
    }
};

// A lane's part of one row of each input, on its way.
template <typename E, int NB, bool GATE, bool BACKWARD>
struct Row {
    Raw<E> x[NB], g[GATE ? NB : 1], dy[BACKWARD ? NB : 1];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            x[i].clear();
            if (GATE) g[i].clear();
            if (BACKWARD) dy[i].clear();
        }
    }
};

// The walk of the inputs, ahead of the work.
template <typename E, int LANES, int NB, bool GATE, bool BACKWARD>
struct Loads {
    Token token;
    Walk x, g;
    long long flat, flat_on;     // dy, contiguous

    __device__ __forceinline__ Loads(const NormArgs &p, int h, unsigned n, unsigned step)
        : token(p, n, step), x(p, n, step, h, p.lay.x_sb, p.lay.x_st, p.lay.x_sh),
          g(p, n, step, h, p.lay.g_sb, p.lay.g_st, p.lay.g_sh),
          flat((static_cast<long long>(n) * p.H + h) * p.d),
          flat_on(static_cast<long long>(step) * p.H * p.d) {}
    __device__ __forceinline__ void next(const NormArgs &p, const Place<LANES, NB> &at,
                                         Row<E, NB, GATE, BACKWARD> &row) {
        if (token.n < p.tokens) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                if (at.there[i]) {
                    row.x[i].load(static_cast<const E *>(p.x) + x.at + at.c[i]);
                    if (GATE) row.g[i].load(static_cast<const E *>(p.gate) + g.at + at.c[i]);
                    if (BACKWARD) row.dy[i].load(static_cast<const E *>(p.dy) + flat + at.c[i]);
                }
        }
        const bool wraps = token.next(p);
        x.next(wraps);
        if (GATE) g.next(wraps);
        if (BACKWARD) flat += flat_on;
    }
};

// x becomes xhat; returns r.
template <int LANES, int NB>
__device__ __forceinline__ float normalise(const NormArgs &p, const Place<LANES, NB> &at,
                                           Pair (&x)[NB][4]) {
    if (p.layer) {
        Pair s = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = add2(s, x[i][e]);
        const Pair mean = twice(-p.inv_d * group_sum<LANES>(s));
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = at.there[i] ? add2(x[i][e], mean) : 0;
    }
    Pair s = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fma2(x[i][e], x[i][e], s);
    const float r = rsqrtf(fmaf(group_sum<LANES>(s), p.inv_d, p.eps));
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = mul2(x[i][e], twice(r));
    return r;
}

template <typename E, int LANES, int NB, bool GATE>
__global__ void __launch_bounds__(32 * kWarps, kFwdPerSm<E, NB>) norm_fwd_kernel(const NormArgs p) {
    const Place<LANES, NB> at(p);
    Pair w[NB][4], b[NB][4];
    load_weights<LANES, NB>(p, at, w, b);
    const unsigned step = gridDim.x / p.groups * kWarps;
    unsigned n = blockIdx.x / p.groups * kWarps + threadIdx.x / 32;
    Loads<E, LANES, NB, GATE, false> loads(p, at.h, n, step);
    Row<E, NB, GATE, false> row, next;   // the next token's loads are on their way
    row.clear();
    next.clear();
    loads.next(p, at, row);
    E *py = static_cast<E *>(p.y) + (static_cast<long long>(n) * p.H + at.h) * p.d;
    for (; n < p.tokens; n += step, py += static_cast<long long>(step) * p.H * p.d) {
        loads.next(p, at, next);
        Pair x[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i) row.x[i].get(x[i]);
        normalise<LANES, NB>(p, at, x);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            Pair m[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = z[e] = fma2(x[i][e], w[i][e], b[i][e]);
            if (GATE) row.g[i].get(z);
            Pair f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = sigmoid(z[e], E{});
            if (p.silu)
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = mul2(f[e], z[e]);
            if (GATE)
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = mul2(f[e], m[e]);
            if (at.there[i]) Raw<E>::store(py + at.c[i], f);
        }
        row = next;
    }
}

// The sums of a block in 64 bits: over its warps in their order, and over the heads of a warp where
// they share a weight.  v: a lane's values, sums of at most kSumRows rows; out: the block's row of
// the partial sums.  Two fp32 numbers hold a sum and what its roundings leave (Knuth's two-sum), which
// is quicker than fp64 additions (B3 T777, 5 heads of 96 in fp32, forward and backward 16.3 us for
// 19.2), but for sums past fp32's range.
template <int LANES, int NB>
__device__ __forceinline__ void block_sums(const NormArgs &p, const Place<LANES, NB> &at,
                                           float (*buf)[32][NB][8], const Pair (&v)[NB][4],
                                           double *out) {
    constexpr int ROWS = 32 / LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();   // the buffer's last use
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) reinterpret_cast<Pair *>(buf[warp][lane][i])[e] = v[i][e];
    __syncthreads();
    // one thread a value: per head [ROWS][d], or summed over the rows [d]
    const int values = p.per_channel ? ROWS * p.d : p.d;
    for (int c = threadIdx.x; c < values; c += 32 * kWarps) {
        const int r = c / p.d, ch = c - r * p.d, i = ch / 8 / LANES, j = ch / 8 % LANES;
        const int rows = p.per_channel ? r + 1 : ROWS;
        float s = 0.f, rest = 0.f;
        for (int row = r; row < rows; ++row)
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float x = buf[k][row * LANES + j][i][ch % 8], sum = s + x, part = sum - s;
                rest += (s - (sum - part)) + (x - part);
                s = sum;
            }
        double total = static_cast<double>(s) + static_cast<double>(rest);
        if (!(fabsf(s) < INFINITY)) {
            total = 0.;
            for (int row = r; row < rows; ++row)
                for (int k = 0; k < kWarps; ++k) total += buf[k][row * LANES + j][i][ch % 8];
        }
        out[c] = total;
    }
}

template <typename E, int LANES, int NB, bool GATE>
__global__ void __launch_bounds__(32 * kWarps, NB == 1 ? 2 : 1) norm_bwd_kernel(const NormArgs p) {
    __shared__ __align__(16) float buf[kWarps][32][NB][8];
    const Place<LANES, NB> at(p);
    Pair w[NB][4], b[NB][4], dw[NB][4], db[NB][4];
    load_weights<LANES, NB>(p, at, w, b);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = db[i][e] = 0;
    const unsigned step = gridDim.x / p.groups * kWarps;
    const unsigned n = blockIdx.x / p.groups * kWarps + threadIdx.x / 32;
    Loads<E, LANES, NB, GATE, true> loads(p, at.h, n, step);
    Token token(p, n, step);
    Walk out(p, n, step, at.h, p.lay.dx_sb, p.lay.dx_st, p.lay.dx_sh);
    Row<E, NB, GATE, true> row, next;   // the next token's loads are on their way
    row.clear();
    next.clear();
    loads.next(p, at, row);
    long long flat = (static_cast<long long>(n) * p.H + at.h) * p.d;
    while (token.n < p.tokens) {
        loads.next(p, at, next);
        Pair x[NB][4], u[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i) row.x[i].get(x[i]);
        const float r = normalise<LANES, NB>(p, at, x);
        Pair su = 0, sux = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            Pair m[4], z[4], dy[4], s[4], f[4];
            row.dy[i].get(dy);
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = z[e] = fma2(x[i][e], w[i][e], b[i][e]);
            if (GATE) row.g[i].get(z);
            // f and, in s, its slope
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = sigmoid(z[e], E{});
                s[e] = fma2(f[e], twice(-1.f), twice(1.f));
            }
            if (p.silu) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[e] = mul2(f[e], fma2(z[e], s[e], twice(1.f)));
                    f[e] = mul2(f[e], z[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = mul2(f[e], s[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Pair dn = mul2(dy[e], GATE ? f[e] : s[e]);
                if (GATE) s[e] = mul2(mul2(dy[e], m[e]), s[e]);
                dw[i][e] = fma2(dn, x[i][e], dw[i][e]);
                db[i][e] = add2(db[i][e], dn);
                u[i][e] = mul2(dn, w[i][e]);
                su = add2(su, u[i][e]);
                sux = fma2(u[i][e], x[i][e], sux);
            }
            if (GATE && at.there[i]) Raw<E>::store(static_cast<E *>(p.dgate) + flat + at.c[i], s);
        }
        const Pair m1 = twice(-p.inv_d * group_sum<LANES>(sux));
        const Pair m0 = twice(p.layer ? -p.inv_d * group_sum<LANES>(su) : 0.f);
        E *pd = static_cast<E *>(p.dx) + out.at;
        out.next(token.next(p));
        flat += static_cast<long long>(step) * p.H * p.d;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                u[i][e] = mul2(twice(r), fma2(x[i][e], m1, add2(u[i][e], m0)));
            if (at.there[i]) Raw<E>::store(pd + at.c[i], u[i]);
        }
        row = next;
    }
    if (p.partial) {
        constexpr int ROWS = 32 / LANES;
        const long long row = p.per_channel ? static_cast<long long>(ROWS) * p.d : p.d;
        double *out = p.partial + blockIdx.x * row;
        block_sums<LANES, NB>(p, at, buf, dw, out);
        block_sums<LANES, NB>(p, at, buf, db, out + gridDim.x * row);
    }
}

// The gradients of weight (blockIdx.y = 0) and bias from the blocks' sums, partial
// [2][blocks][values]: the values of blocks b, b + groups, ... belong to the same heads where
// each head has weights of its own (groups > 1 only there), else every block has the same ones.
// 32 channels of a block, one warp-wide row of 32 partial sums each; sums in fp64.
__global__ void __launch_bounds__(1024) reduce_kernel(const double *partial, unsigned blocks,
                                                      int groups, int values, int channels,
                                                      float *dw, float *db) {
    __shared__ double buf[32][33];
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    double s = 0.;
    if (c < channels) {
        const unsigned group = c / values;
        const double *from = partial + static_cast<size_t>(blockIdx.y) * blocks * values + c % values;
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
long long token_blocks(long long tokens, int groups, long long most, int sum_rows) {
    const long long want = std::min((tokens + kWarps - 1) / kWarps, std::max(1LL, most / groups));
    return std::max(want, sum_rows ? (tokens + kWarps * sum_rows - 1) / (kWarps * sum_rows) : 1);
}

template <typename E, int LANES, int NB>
int launch_fwd(const NormArgs &a, int sms, cudaStream_t stream) {
    const long long tb = token_blocks(a.tokens, a.groups, sms * kFwdPerSm<E, NB>, 0);
    if (tb * a.groups > INT_MAX) return -1;
    const unsigned grid = static_cast<unsigned>(tb * a.groups);
    if (a.gate) norm_fwd_kernel<E, LANES, NB, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else norm_fwd_kernel<E, LANES, NB, false><<<grid, 32 * kWarps, 0, stream>>>(a);
    return static_cast<int>(cudaGetLastError());
}

template <typename E, int LANES, int NB>
int launch_bwd(const NormArgs &a, float *dw, float *db, cudaStream_t stream) {
    const long long tb = token_blocks(a.tokens, a.groups, kBwdBlocks, kSumRows);
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
int fwd(const NormArgs &a, int sms, cudaStream_t stream) {
    if (a.d <= 64) return launch_fwd<E, 8, 1>(a, sms, stream);
    if (a.d <= 128) return launch_fwd<E, 16, 1>(a, sms, stream);
    if (a.d <= 256) return launch_fwd<E, 32, 1>(a, sms, stream);
    return launch_fwd<E, 32, 2>(a, sms, stream);
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
    if (backward) {
        for (long long s : {lay.dx_sb, lay.dx_st, lay.dx_sh})
            if (s < 0 || s % 8) return GLA_ERR_ARG;
        // x may be spread out from one row; its gradient is a row for each
        if ((B > 1 && !lay.dx_sb) || (T > 1 && !lay.dx_st) || (H > 1 && !lay.dx_sh))
            return GLA_ERR_ARG;
    }
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

// The memory of x, gate, weight and bias, in this order.
void inputs_of(Span (&in)[4], const NormArgs &a, int B, int T, const gla_norm_act_layout &lay,
               int size) {
    const auto reach = [&](long long sb, long long st, long long sh) {
        return static_cast<unsigned long long>((B - 1) * sb + (T - 1) * st + (a.H - 1) * sh + a.d);
    };
    const unsigned long long weights = a.per_channel ? static_cast<unsigned long long>(a.H) * a.d : a.d;
    in[0] = span_of(a.x, reach(lay.x_sb, lay.x_st, lay.x_sh), size);
    in[1] = span_of(a.gate, reach(lay.g_sb, lay.g_st, lay.g_sh), size);
    in[2] = span_of(a.w, weights, 4);
    in[3] = span_of(a.b, weights, 4);
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
    const int size = options->dtype == GLA_BF16 ? 2 : 4;
    Span in[4];
    inputs_of(in, a, B, T, *layout, size);
    if (meets_any(span_of(y, static_cast<unsigned long long>(a.tokens) * H * d, size), in))
        return GLA_ERR_ARG;
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const int e = options->dtype == GLA_BF16 ? fwd<__nv_bfloat16>(a, sms, stream)
                                             : fwd<float>(a, sms, stream);
    return e == 0 ? GLA_OK : e < 0 ? GLA_ERR_ARG : GLA_ERR_LAUNCH;
}

unsigned long gla_group_norm_act_bwd_scratch(int B, int T, int H, int d) {
    using namespace gla;
    if (B <= 0 || T <= 0 || H <= 0 || d <= 0) return 0;
    const int rows = rows_of(d), groups = (H + rows - 1) / rows;
    const long long tb = token_blocks(static_cast<long long>(B) * T, groups, kBwdBlocks, kSumRows);
    return 2ul * sizeof(double) * tb * groups * rows * d;
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
        a.partial = static_cast<double *>(scratch);
    }
    const int size = options->dtype == GLA_BF16 ? 2 : 4;
    const unsigned long long n = static_cast<unsigned long long>(a.tokens) * H * d;
    const unsigned long long weights =
        options->per_channel ? static_cast<unsigned long long>(H) * d : d;
    const unsigned long long reach = static_cast<unsigned long long>(
        (B - 1) * layout->dx_sb + (T - 1) * layout->dx_st + (H - 1) * layout->dx_sh + d);
    Span in[4];
    inputs_of(in, a, B, T, *layout, size);
    const Span up = span_of(dy, n, size);
    const Span outs[4] = {span_of(grad_x, reach, size), span_of(grad_gate, n, size),
                          span_of(grad_weight, weights, 4), span_of(grad_bias, weights, 4)};
    for (int i = 0; i < 4; ++i) {
        if (meets_any(outs[i], in) || meet(outs[i], up)) return GLA_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return GLA_ERR_ARG;
    }
    int sms = 0;
    st = usable_device(&sms);
    if (st != GLA_OK) return st;
    const Span work = span_of(a.partial, gla_group_norm_act_bwd_scratch(B, T, H, d), 1);
    if (meets_any(work, in) || meet(work, up) || meets_any(work, outs)) return GLA_ERR_ARG;
    const int e = options->dtype == GLA_BF16
                      ? bwd<__nv_bfloat16>(a, grad_weight, grad_bias, stream)
                      : bwd<float>(a, grad_weight, grad_bias, stream);
    return e == 0 ? GLA_OK : e < 0 ? GLA_ERR_ARG : GLA_ERR_LAUNCH;
}

}  // extern "C"
