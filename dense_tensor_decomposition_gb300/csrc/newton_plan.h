// How the products of the orthogonalisation are dealt out: host and device code without CUDA, so
// that the rules can be walked over all sizes on any machine.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define MK_HOST_DEVICE __host__ __device__
#else
#define MK_HOST_DEVICE
#endif

namespace mk {

constexpr int kTable = 32;                  // list elements a group of launches

// Matrices of one list element.  Tiles of one matrix, hi and lo of each: X twice (a step
// reads one and writes the other), S, P.
struct Shape {
    int base;                   // first tile
    int rows, cols, count;
    uint32_t first[2];          // number of the first work item: of S and S S, of P X
};
MK_HOST_DEVICE inline int tiles_of(int n) { return (n + 63) / 64; }

// what a launch computes: S, P (from S S), P X, and the last P X, whose result goes to the caller
enum Phase { kGram, kSquare, kUpdate, kResult };
MK_HOST_DEVICE constexpr bool is_update(int phase) { return phase >= kUpdate; }

struct Grid {
    int rt, ct, mt;             // tiles of 64 along rows, columns and the smaller side
    bool wide;
    MK_HOST_DEVICE explicit Grid(const Shape& s)
        : rt(tiles_of(s.rows)), ct(tiles_of(s.cols)), mt(s.rows <= s.cols ? rt : ct), wide(s.rows <= s.cols) {}
    MK_HOST_DEVICE int x(int which) const { return 2 * which * rt * ct; }
    MK_HOST_DEVICE int x_lo() const { return rt * ct; }
    MK_HOST_DEVICE int s() const { return 4 * rt * ct; }
    MK_HOST_DEVICE int p() const { return s() + 2 * mt * mt; }
    MK_HOST_DEVICE int s_lo() const { return mt * mt; }
    MK_HOST_DEVICE int tiles() const { return 4 * (rt * ct + mt * mt); }
    // contraction indices of a product, in steps of 64
    MK_HOST_DEVICE int steps(int phase) const { return phase != kGram ? mt : wide ? ct : rt; }
};

// Work items of a symmetric result of nb x nb blocks: rows of blocks from the block of 256 they are in on.
MK_HOST_DEVICE inline int symmetric_items(int nb, int ctas) {
    if (ctas == 2) return nb * (nb + 1) / 2;
    const int pairs = nb / 2;           // rows 2 p and 2 p + 1 have nb - 2 p items each
    return pairs * (2 * nb - 2 * pairs + 2) + (nb % 2);
}

// the first of an item's steps that share number `share` of `split` takes
MK_HOST_DEVICE inline int share_begin(int steps, int share, int split) { return steps * share / split; }

// Numbers the work items of a product whose CTAs (or pairs) take blocks of 128 (256) a side, and
// says how long it takes, in microseconds without the launch: waves of items, whose epilogues run
// beside the next one's MMAs.  Steps of 64 indices and epilogues as measured on 12 x 1024 x 4096,
// 2 x 4096 x 4096 and 3 x 512 x 2000; a pair's items are four times a CTA's.
constexpr float kExchange = 2.5f;       // microseconds that a cluster takes to add up its parts of S

// P: n and shape[n] are given, items and split are found
template <typename P>
float number_items(P& p, int phase, int ctas, bool full, int sms) {
    const int f = is_update(phase) ? 1 : 0, block = 2 * ctas;
    const float step = full ? (ctas == 2 ? 1.02f : 0.72f) : f ? (ctas == 2 ? 0.61f : 0.52f) : (ctas == 2 ? 0.33f : 0.26f);
    const float end = (phase == kSquare ? (ctas == 2 ? 8.f : 4.f) : (ctas == 2 ? 4.f : 2.f));
    auto blocks = [&](int tiles) { return (tiles + block - 1) / block; };
    float work = 0.f, longest = 0.f;
    int fewest = INT32_MAX;             // steps of any item
    p.items = 0;
    for (int i = 0; i < p.n; ++i) {
        Shape& s = p.shape[i];
        const Grid g(s);
        s.first[f] = p.items;
        const int64_t items = s.count * (f ? (int64_t)blocks(g.rt) * blocks(g.ct) : (int64_t)symmetric_items(blocks(g.mt), ctas));
        const float one = std::max((float)g.steps(phase) * step, end);
        work += (float)items * one;
        longest = std::max(longest, one);
        fewest = std::min(fewest, g.steps(phase));
        p.items += (uint32_t)items;
    }
    // S by single CTAs, where they are fewer than half of the SMs: two or four an item, with steps
    // enough each for the longest to pay, and one at least for the shortest
    p.split = 1;
    if (phase == kGram && ctas == 1)
        while (p.split < 4 && p.split * 2 <= fewest && p.items * p.split * 2 <= (uint32_t)sms &&
               longest / (2 * p.split) > kExchange)
            p.split *= 2;
    const float units = (float)(sms / ctas), waves = std::ceil((float)p.items / units);
    if (p.split > 1) return longest / (float)p.split + kExchange + end;
    return std::max(longest, waves * work / (float)p.items) + end;
}

// Deals a list's matrices out to launches of at most `elements` parts of list elements and `most` matrices
// together.  count(k): matrices of element k, of n.  take(part, k, b0, matrices, before): the part that holds
// those of element k from b0 on, behind `before` others of the launch.  launch(parts, matrices): whether to go on.
template <typename Count, typename Take, typename Launch>
void deal(int n, int elements, int64_t most, Count count, Take take, Launch launch) {
    int parts = 0;
    int64_t used = 0;
    for (int k = 0; k < n; ++k)
        for (int64_t b = 0, all = count(k); b < all;) {
            if (parts == elements || used == most) {
                if (!launch(parts, used)) return;
                parts = 0;
                used = 0;
            }
            const int64_t here = std::min(all - b, most - used);
            take(parts++, k, b, here, used);
            used += here;
            b += here;
        }
    if (parts > 0) launch(parts, used);
}

}  // namespace mk
