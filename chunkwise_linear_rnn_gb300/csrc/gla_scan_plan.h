/*
 * gla_scan_plan.h — how a scan's work is laid out: tile shape, blocks of a cluster, or a
 * thread's own walk.  Host arithmetic only: no CUDA call, and nothing but the sizes decides.
 */
#pragma once

#include <algorithm>
#include <cmath>
#include <iterator>

namespace gla {

constexpr int kMaxCluster = 16;
// Tokens that a thread of its own walk has on their way at a time.
constexpr int kChunk = 8;

// Blocks of a cluster of blocks of so many channels, at most.
constexpr int cluster_of(int channels) { return channels == 32 ? kMaxCluster : 1; }

// The tiles' ways to the registers: by TMA, where rows are whole 16-byte pieces; four
// neighbouring bf16 channels a thread without it; one.  (B2 T16384, bf16 forward: D2048 by TMA
// 89 us, D2052 by fours 110, D2050 by ones 163.)
enum class Way { kTma, kFour, kOne };

// Channels of a thread block and blocks of a cluster.
struct Choice {
    int width, cluster;
};
// Only narrow blocks stand side by side in time: a cluster of wider ones takes the tokens at a
// time of a longer one of narrow ones, and no less time.
constexpr Choice kChoices[] = {{32, 1}, {32, 2}, {32, 4}, {32, 8}, {32, 16},
                               {64, 1}, {128, 1}};   // the wide ones: forward by TMA

// A launch's work: tokens of the longest sequence and of all, sequences, heads, channels.
struct Work {
    double longest, total, nseq, heads;
    int D, size;             // size: bytes of a value of x
    bool backward;
    Way way;
};

// The time of a launch in us, as far as it takes to choose: how long a block takes for a tile
// (`alone` on its SM, or one of two there; or HBM's rate shared by all that run), times the
// tiles, times the waves.  The figures are fits to 55 shapes, forward and backward, with
// every choice measured; over 70 others the choices made were 1.5% slower than the best on
// average, 24% at most.  (Forward, bf16, us, as channels x cluster: B8 T2048 D2048 128x1 47,
// 64x1 42, 32x1 46, 32x2 55; B16 T512 D2048 128x1 24, 64x1 27; B1 T262144 D1024 32x4 466, 32x8 333, 32x16 444; B2 T143060 D176
// 32x8 131, 32x16 95; fp32 B7 T458 D1360 64x1 14, 32x1 12; fp32 16 ragged sequences of 20000
// tokens, D1024, 32x4 59, 32x1 47.)
inline double estimate(const Work &k, Choice c, int sms) {
    const int run = k.way == Way::kTma ? 4096 / c.width : k.way == Way::kFour ? 128 : 64;
    const double tokens = run * c.cluster;
    const double blocks = k.nseq * k.heads * ((k.D + c.width - 1) / c.width) * c.cluster;
    // blocks that run alone on an SM, and at once: large clusters do not fill every part of the chip
    const double one = sms * (c.cluster < 8 ? 1.0 : 0.72);
    const bool single = k.backward && (k.way == Way::kFour || (k.way == Way::kTma && k.size == 4));
    const double most = single ? one : sms * (c.cluster < 8 ? 2.0 : c.cluster == 8 ? 1.9 : 1.35);
    double alone, two;
    if (k.way == Way::kTma) {
        alone = k.backward ? 1.4 : 1.0;
        two = k.backward ? 2.2 : 0.4 * (k.size + 2);
    } else if (k.way == Way::kFour) {
        alone = k.backward ? 1.5 : 1.1;
        two = 1.6;   // the backward's blocks are always alone
    } else {
        alone = k.backward ? 1.5 : 0.9;
        two = k.backward ? 2.4 : 1.4;
    }
    if (c.cluster > 1) alone *= 1.4;
    const double bytes = run * c.width * (k.backward ? 8 + 3 * k.size : 4 + 2 * k.size) / 6.5e6;
    const auto tile = [&](double n) { return std::max(n <= one ? alone : two, n * bytes); };
    const double begin = 1.5 + (c.cluster > 1 ? 0.18 * c.cluster : 0.0);
    const double tiles = std::ceil(k.longest / tokens);
    if (k.nseq == 1) {
        const double waves = std::floor(blocks / most), rest = blocks - waves * most;
        return waves * (tiles * tile(most) + begin) + (rest > 0 ? tiles * tile(rest) + begin : 0.0);
    }
    // the longest sequence, or all of them shared by the blocks that run at once
    const double n = std::min(blocks, most), first = tiles * alone + begin;
    const double all = blocks / n * ((k.total / k.nseq / tokens + 0.5) * tile(n) + begin);
    return std::max(first, all) + 0.25 * std::min(first, all);
}

// The same for threads that walk a sequence each: a chunk after another, and HBM's rate.
// (us, bf16, walks / tiles: forward B256 T1 D4096 10 / 59, B64 T64 D4096 28 / 32, B64 T256 D4096
// 104 / 84, B1 T64 D2048 7.1 / 3.4; backward B256 T16 D4096 53 / 306, B64 T100 D4096 87 / 102,
// B64 T400 D4096 329 / 272.  Over 190 shapes the faster of both but for 0.6% on average, 30% at most.)
inline double walk_time(const Work &k) {
    const double chunks = std::ceil(k.longest / kChunk);
    const double bytes = k.heads * k.total * k.D * (k.backward ? 8 + 3 * k.size : 4 + 2 * k.size);
    return 1.0 + chunks * (k.backward ? 1.35 : 0.55) + bytes * (k.backward ? 1.2 : 1.0) / 6.5e6;
}

// What a launch does: threads that walk a sequence each, or blocks of this shape.
struct Layout {
    bool walk;
    Choice tiles;
};

inline Layout layout(const Work &k, int sms) {
    const int count = k.way == Way::kTma && !k.backward ? static_cast<int>(std::size(kChoices)) : 5;
    Layout l = {false, kChoices[0]};
    double least = estimate(k, kChoices[0], sms);
    for (int i = 1; i < count; ++i) {
        const double t = estimate(k, kChoices[i], sms);
        if (t >= least) continue;
        least = t;
        l.tiles = kChoices[i];
    }
    // a grid of 64 threads a block, one to every 4 channels or one
    const double threads = k.nseq * k.heads * (k.way == Way::kOne ? k.D : k.D / 4);
    // (empty sequences alone always walk: there is nothing that TMA could point at)
    l.walk = (k.longest == 0 || least >= walk_time(k)) && threads < 0x7fffff00;
    return l;
}

}  // namespace gla
