// Sums of rows over the tokens that point to them: for every row of a table a term of
// each of its tokens is added, in the order of the tokens, so that results repeat bit
// by bit.  Two ways:
//   * few tokens (own_kernel): one launch.  Every CTA owns some of the rows, finds the
//     tokens that point to them, groups them by row and writes its rows, zeros included.
//   * many tokens: the tokens are sorted by row (sort.cu), and CTAs walk the sorted
//     tokens in tiles of equal length, however long a row's run of tokens is, and set
//     rows without tokens to zero (row_sum_kernel); runs that cross tile borders are
//     joined by a last launch (join_kernel).
// Both add with sum_list(), which splits a list of sorted tokens over groups of lanes
// and joins the runs that cross the groups' borders.
#pragma once

#include "rows.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- sums over a list of sorted tokens

template <typename TO, int VEC>
__device__ __forceinline__ void write_row(const RowSumArgs& a, int m, uint32_t v, int64_t col, const float* acc) {
    Pack<TO, VEC>* p = reinterpret_cast<Pack<TO, VEC>*>(static_cast<TO*>(a.out[m]) + (int64_t)v * a.out_stride + col);
    Pack<TO, VEC> x;
    if (a.accumulate) x = *p;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float s = a.scale * acc[e];
        x.v[e] = from_f32<TO>(a.accumulate ? to_f32(x.v[e]) + s : s);
    }
    *p = x;
}

// What lies around a list: whether its first run began before it, whether its last
// one goes on after it, and where such runs' sums go (indexed by column).
struct Around {
    bool before, after;
    float* head;
    float* tail;
};

// Adds the terms of a list of `count` >= 1 tokens sorted by row over the columns from
// col0 on, and writes the finished rows.  list(p): entry p, its row first (.x).  A group
// of L = 2^log2L threads (of kN in all, which sync() makes wait for one another) walks
// count / groups consecutive tokens; a lane has VEC columns.  A run that crosses groups
// is finished by the group in which it began, from the other groups' parts in `heads`
// (kN * VEC floats), in the order of the groups.
//
// Terms<List> terms(context, list, p0, p1, col) gives a lane the terms of tokens p0 .. p1,
// kB at a time: after load(p), key(j) is the row of token p + j and add(j, acc) adds its
// term; behind p1 these repeat some token of the list.  Lanes behind the last column
// take part only where the terms need all lanes of a group (kAllLanes).
//
// kRagged: a lane's last columns may lie behind the width, and rows start anywhere, so
// that results are written one column at a time.
template <typename TO, int VEC, template <typename> typename Terms, int kN, bool kRagged = false, typename Context,
          typename List, typename Row, typename Sync>
__device__ __forceinline__ void sum_list(const RowSumArgs& a, int m, const Context& context, const List& list,
                                         const Row& row_of, int count, int log2L, int64_t col0, float* heads,
                                         const Around& around, const Sync& sync) {
    constexpr int B = Terms<List>::kB;
    const int L = 1 << log2L, groups = kN >> log2L;
    const int group = threadIdx.x >> log2L, lane = threadIdx.x & (L - 1);
    const int64_t col = col0 + lane * VEC;
    const bool on = col < a.width;
    const bool part = on || Terms<List>::kAllLanes;
    const int share = (count + groups - 1) / groups;
    const int p0 = group * share < count ? group * share : count;
    const int p1 = p0 + share < count ? p0 + share : count;
    float acc[VEC];
    auto put = [&](float* dst) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) dst[e] = acc[e];
    };
    auto add = [&](const float* src) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += src[e];
    };
    float* own_head = heads + (size_t)threadIdx.x * VEC;
    uint32_t cur = 0;
    bool open = false;          // the run at the end began in this group and goes on
    auto finish = [&]() {
        if constexpr (kRagged) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (col + e < a.width) write_row<TO, 1>(a, m, row_of(cur), col + e, acc + e);
        } else {
            if (on) write_row<TO, VEC>(a, m, row_of(cur), col, acc);
        }
    };
    auto put_part = [&](float* row) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (!kRagged || col + e < a.width) row[col + e] = acc[e];
    };
    if (p0 < p1 && part) {
        cur = list(p0).x;
        bool began_before = p0 > 0 ? list(p0 - 1).x == cur : around.before;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
        Terms<List> terms(context, list, p0, p1, col);
        for (int p = p0; p < p1; p += B) {
            terms.load(p);
            if (p + B <= p1 && terms.key(B - 1) == cur) {       // all of one row
#pragma unroll
                for (int j = 0; j < B; ++j) terms.add(j, acc);
                continue;
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (p + j < p1) {
                    if (terms.key(j) != cur) {
                        if (began_before) put(own_head);
                        else finish();
                        began_before = false;
                        cur = terms.key(j);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
                    }
                    terms.add(j, acc);
                }
            }
        }
        const bool goes_on = p1 < count ? list(p1).x == cur : around.after;
        if (began_before) put(own_head);
        else if (goes_on) open = true;
        else finish();
    }
    sync();
    if (!on) return;
    if (open) {
        int g = group + 1;
        for (; g * share < count && list(g * share).x == cur; ++g) add(heads + ((size_t)(g << log2L) + lane) * VEC);
        if (g * share >= count && around.after && list(count - 1).x == cur) put_part(around.tail);
        else finish();
    }
    if (group == 0 && around.before) {
        const uint32_t first = list(0).x;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = own_head[e];
        for (int g = 1; g * share < count && list(g * share).x == first; ++g)
            add(heads + ((size_t)(g << log2L) + lane) * VEC);
        put_part(around.head);
    }
}

// Zeros for those of `rows` local rows, from local row r0 on, that no token points
// to, by one warp; row_of gives a local row's number in the table (kNone: none).  Rows at
// any offset are written in 16-byte vectors but for their ends (3000 tokens into 200000
// rows of 33 16-bit columns: 38 us by single columns, 12 so).
template <typename TO, int VEC, typename Touched, typename Row>
__device__ __forceinline__ void zero_rows(const RowSumArgs& a, int m, uint32_t r0, uint32_t rows, int64_t col0,
                                          uint32_t vecs, const Touched& touched, const Row& row_of) {
    const uint32_t lane = threadIdx.x & 31;
    Pack<TO, VEC> zero;
#pragma unroll
    for (int e = 0; e < VEC; ++e) zero.v[e] = from_f32<TO>(0.f);
    auto at = [&](uint32_t v) {
        return reinterpret_cast<Pack<TO, VEC>*>(static_cast<TO*>(a.out[m]) + (int64_t)v * a.out_stride + col0);
    };
    if (vecs >= 8) {
        // by as many lanes as a row has of them
        constexpr uint32_t kPer = sizeof(zero) < 16 ? 16 / sizeof(zero) : 1, kWide = sizeof(zero) * kPer / 16;
        const uint32_t wide = vecs / kPer * kWide, lanes = wide > 16 ? 32 : wide > 8 ? 16 : 8;
        const uint32_t l = lane & (lanes - 1);
        for (uint32_t r = r0 + lane / lanes; r < r0 + rows; r += 32 / lanes) {
            const uint32_t v = touched(r) ? kNone : row_of(r);
            if (v == kNone) continue;
            Pack<TO, VEC>* dst = at(v);
            const uint32_t skew = (uint32_t)(reinterpret_cast<uintptr_t>(dst) / sizeof(zero)) % kPer;
            const uint32_t head = (kPer - skew) % kPer, body = (vecs - head) / kPer, tail = (vecs - head) % kPer;
            if (l < head) dst[l] = zero;
            if (l < tail) dst[vecs - tail + l] = zero;
            uint4* mid = reinterpret_cast<uint4*>(dst + head);
#pragma unroll 4
            for (uint32_t c = l; c < body * kWide; c += lanes) mid[c] = make_uint4(0u, 0u, 0u, 0u);
        }
    } else {
        for (uint32_t i = lane; i < rows * vecs; i += 32) {
            const uint32_t r = i / vecs, v = touched(r0 + r) ? kNone : row_of(r0 + r);
            if (v != kNone) at(v)[i - r * vecs] = zero;
        }
    }
}

// 32 rows of a warp from r0 on: a lane looks one of them up among the sorted tokens,
// then those without tokens become zero
template <typename TO, int VEC, typename Key>
__device__ __forceinline__ void zero_unsorted_rows(const RowSumArgs& a, int m, int64_t r0, const Key& key) {
    const int64_t n = a.index.n, rows = a.index.rows[m], v = r0 + (threadIdx.x & 31);
    if (r0 >= rows) return;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (key(mid) < v) lo = mid + 1;
        else hi = mid;
    }
    const bool has = v >= rows || (lo < n && key(lo) == (uint32_t)v);
    const uint32_t touched = __ballot_sync(0xFFFFFFFFu, has);
    if (touched == 0xFFFFFFFFu) return;
    zero_rows<TO, VEC>(
        a, m, 0, 32, 0, (uint32_t)(a.width / VEC), [&](uint32_t r) { return (touched >> r & 1u) != 0; },
        [&](uint32_t r) { return (uint32_t)(r0 + r); });
}

// what the terms of (row, token) entries are made from
struct TermsOf {
    const RowSumArgs& a;
    int m;
};

// ---------------------------------------------------------------- few tokens: one launch

constexpr int kOwnThreads = 1024;
constexpr int kOwnWarps = kOwnThreads / 32;
constexpr int kSumThreads = 512;        // of which these group and add (2^9 lanes), while the others write zeros
constexpr int kSumWarps = kSumThreads / 32;
// The most tokens for which two lists of 4 bytes a token fit into a CTA's shared memory
// beside the sums' own.  Up to there one launch is faster than sorting first unless few
// rows have most of the tokens, at which the rule does not look (16384 tokens, this way
// and sorted first: into 512 rows of 256 fp32 12.3 and 18.5 us, 20000 of 128 bf16 12.2 and
// 26.7; samples of a 256^3 model, R = 64, 20.3 and 24.7; but u^3 over 2000 rows of 1024 bf16
// 34.6 and 28.4, and a 512 x 512 x 1 model, R = 128, whose one row is a single CTA's, 368
// and 31).
constexpr int kTokenBits = 14;
constexpr int kOwnTokens = 1 << kTokenBits;
constexpr int kOwnRows = 1 << 13;       // rows of a CTA

// Owners: blocks of 2^row_shift consecutive rows go to the CTAs (blockIdx.x) in turn,
// so that frequent rows, which often have small numbers, are spread.
struct OwnArgs {
    RowSumArgs a;
    int row_shift;
    uint32_t owned;         // most rows a CTA owns
    uint32_t per_warp;      // tokens that a warp looks at
    int log2L;
    int64_t part;           // columns of a CTA (blockIdx.y)
    uint32_t first_bytes;   // of shared memory, for `list` and then the terms
};

// Bound by memory: the rows' writes, most of them zeros where tokens are few, and the
// terms' reads; for the smallest, by latencies: 4096 samples of a 256^3 model take about
// 2 us to look through, 2 to group, 2.5 to add.  The zeros begin before it is known which
// rows have tokens: while one half of the CTA groups the tokens, the other writes them to
// all rows, from the last one on; rows with tokens are written again.
template <typename TO, int VEC, template <typename> typename Terms>
__global__ void __launch_bounds__(kOwnThreads, 1) own_kernel(const __grid_constant__ OwnArgs o) {
    extern __shared__ float4 own_smem[];
    after_previous();
    const RowSumArgs& a = o.a;
    uint32_t* list = reinterpret_cast<uint32_t*>(own_smem);                     // tokens of the CTA's rows; then the terms'
    float* heads = reinterpret_cast<float*>(reinterpret_cast<char*>(own_smem) + o.first_bytes);     // kSumThreads * VEC
    uint32_t* cursor = reinterpret_cast<uint32_t*>(heads + kSumThreads * VEC);  // owned: tokens of each row, then their places
    uint32_t* touched = cursor + o.owned;                                       // a bit for each owned row
    uint32_t* found = touched + (o.owned + 31) / 32;                            // the same with gaps, a part a warp; then sorted
    __shared__ uint32_t warp_found[kOwnWarps], sums[kSumWarps], tokens, next_unit, last_unit;
    __shared__ volatile int grouped;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.z;
    const uint32_t G = gridDim.x, n = (uint32_t)a.index.n, rows = (uint32_t)a.index.rows[m];
    const uint32_t low = (1u << o.row_shift) - 1;
    auto row_of = [&](uint32_t r) -> uint32_t {
        const uint64_t v = (((uint64_t)(r >> o.row_shift) * G + blockIdx.x) << o.row_shift) | (r & low);
        return r < o.owned && v < rows ? (uint32_t)v : kNone;
    };
    auto sync = [] { asm volatile("barrier.sync 1, %0;" ::"n"(kSumThreads) : "memory"); };
    // zeros are written a unit of rows at a time
    const int64_t col0 = (int64_t)blockIdx.y * o.part;
    const uint32_t vecs = (uint32_t)((a.width - col0 < o.part ? a.width - col0 : o.part) / VEC);
    const uint32_t unit = vecs >= 512 ? 1 : 512 / vecs, units = (o.owned + unit - 1) / unit;
    auto take = [&](uint32_t* counter) {
        uint32_t u = 0;
        if (lane == 0) u = atomicAdd(counter, 1u);
        return __shfl_sync(0xFFFFFFFFu, u, 0);
    };

    // the CTA's tokens, as (owned row, token), in order in every warp's part
    for (uint32_t i = threadIdx.x; i < o.owned; i += kOwnThreads) cursor[i] = 0;
    if (threadIdx.x == 0) {
        next_unit = 0;
        last_unit = 0;
        grouped = 0;
    }
    __syncthreads();
    uint32_t count = 0;
    with_key(a.index, [&](auto key_of) {
        constexpr int kLook = decltype(key_of)::kLook;      // tokens a lane looks up at once
        for (uint32_t k0 = 0; k0 < o.per_warp; k0 += kLook * 32) {
            uint32_t key[kLook];
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                const uint32_t k = k0 + u * 32 + lane, t = warp * o.per_warp + k;
                key[u] = k < o.per_warp && t < n ? key_of(a.index, t, m) : kNone;
            }
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                const uint32_t t = warp * o.per_warp + k0 + u * 32 + lane, v = key[u];
                const uint32_t block = v >> o.row_shift, turn = block / G;
                const bool mine = v != kNone && block - turn * G == blockIdx.x;
                const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, mine);
                if (mine) {
                    const uint32_t r = (turn << o.row_shift) | (v & low);
                    found[warp * o.per_warp + count + __popc(ballot & ((1u << lane) - 1))] = (r << kTokenBits) | t;
                    atomicAdd(cursor + r, 1u);
                }
                count += __popc(ballot);
            }
        }
    });
    if (lane == 0) warp_found[warp] = count;
    __syncthreads();
    if (warp < kSumWarps) {
        // gaps out; the counts become the rows' first places
        const uint32_t c = warp_found[lane];
        uint32_t upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += up;
        }
        const uint32_t total = __shfl_sync(0xFFFFFFFFu, upto, 31);
        for (int w = warp; w < kOwnWarps; w += kSumWarps) {
            const uint32_t size = __shfl_sync(0xFFFFFFFFu, c, w), base = __shfl_sync(0xFFFFFFFFu, upto - c, w);
            for (uint32_t k = lane; k < size; k += 32) list[base + k] = found[w * o.per_warp + k];
        }
        const uint32_t per = (o.owned + kSumThreads - 1) / kSumThreads;
        uint32_t mine = 0, all;
        for (uint32_t k = 0; k < per; ++k) {
            const uint32_t r = threadIdx.x * per + k;
            mine += r < o.owned ? cursor[r] : 0;
        }
        uint32_t at = scan_warps<kSumWarps>(mine, sums, all, sync);
        for (uint32_t r = threadIdx.x; r < (o.owned + 31) / 32 * 32; r += kSumThreads) {
            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, r < o.owned && cursor[r] != 0);
            if (lane == 0) touched[r / 32] = bits;
        }
        sync();
        for (uint32_t k = 0; k < per; ++k) {
            const uint32_t r = threadIdx.x * per + k;
            if (r >= o.owned) break;
            const uint32_t c = cursor[r];
            cursor[r] = at;
            at += c;
        }
        sync();
        // in order of the tokens within each row
        if (total <= kSumThreads) {
            // few: every thread counts the tokens of its row that come before its own
            if (threadIdx.x < total) {
                const uint32_t x = list[threadIdx.x], r = x >> kTokenBits;
                uint32_t before = 0;
#pragma unroll 8
                for (uint32_t k = 0; k < threadIdx.x; ++k) before += list[k] >> kTokenBits == r;
                found[cursor[r] + before] = x;
            }
            sync();
        } else if (warp == 0) {
            // one warp places them 32 at a time
            for (uint32_t k = 0; k < total; k += 32) {
                const uint32_t x = k + lane < total ? list[k + lane] : kNone;
                const uint32_t r = x >> kTokenBits;
                const uint32_t peers = __match_any_sync(0xFFFFFFFFu, r);
                uint32_t to = 0;
                if (k + lane < total) to = cursor[r] + __popc(peers & ((1u << lane) - 1));
                __syncwarp();
                if (k + lane < total) {
                    found[to] = x;
                    if ((peers >> lane) == 1u) cursor[r] = to + 1;      // the last of its row
                }
                __syncwarp();
            }
        }
        if (threadIdx.x == 0) {
            tokens = total;
            grouped = 1;
        }
    } else if (!a.accumulate) {
        while (!grouped) {
            const uint32_t u = take(&last_unit);
            if (u >= units) break;
            zero_rows<TO, VEC>(a, m, (units - 1 - u) * unit, unit, col0, vecs, [](uint32_t) { return false; }, row_of);
        }
    }
    __syncthreads();
    const uint32_t left = units - (last_unit < units ? last_unit : units);
    const int total = (int)tokens;
    if (warp < kSumWarps && total > 0) {
        auto at_place = [&](int p) { return make_uint2(found[p] >> kTokenBits, found[p] & (kOwnTokens - 1)); };
        sum_list<TO, VEC, Terms, kSumThreads>(a, m, TermsOf{a, m}, at_place, row_of, total, o.log2L, col0, heads,
                                              Around{false, false, nullptr, nullptr}, sync);
    }
    if (a.accumulate) return;
    auto is_touched = [&](uint32_t r) { return r >= o.owned || (touched[r >> 5] >> (r & 31) & 1u) != 0; };
    for (uint32_t u = take(&next_unit); u < left; u = take(&next_unit))
        zero_rows<TO, VEC>(a, m, u * unit, unit, col0, vecs, is_touched, row_of);
}

// ---------------------------------------------------------------- many tokens

constexpr int kTile = kThreads;         // most sorted tokens of a CTA of row_sum_kernel

// sorted tokens of a CTA: fewer where the GPU would not have two CTAs an SM
inline int64_t tile_tokens(int64_t n) {
    return n >= 2 * kSms * kTile ? kTile : n >= kSms * kTile ? kTile / 2 : kTile / 4;
}

struct SumArgs {
    RowSumArgs a;
    Sorted sorted;
    float* part;            // d x tiles x 2 x width: sums of the tile's first run that began before, of its last that goes on
    int64_t tile;           // tokens of a tile
    int64_t tiles;
    int log2L;
    int64_t columns;        // columns of a CTA (blockIdx.y)
};

__device__ __forceinline__ uint32_t key_at(const SumArgs& s, int m, int64_t p) {
    return *reinterpret_cast<const uint32_t*>(s.sorted.entries + (m * s.a.index.n + p) * s.sorted.bytes);
}

// The first s.tiles CTAs (blockIdx.x) have a tile of the sorted tokens each; those
// behind write zeros, 32 rows a warp.
template <typename TO, int VEC, template <typename> typename Terms>
__global__ void __launch_bounds__(kThreads) row_sum_kernel(const __grid_constant__ SumArgs s) {
    __shared__ uint2 pairs[kTile];
    __shared__ float4 heads[(kThreads * VEC + 3) / 4];
    after_previous();
    const RowSumArgs& a = s.a;
    const int m = blockIdx.z;
    const int64_t n = a.index.n;
    if (blockIdx.x >= s.tiles) {
        if (blockIdx.y > 0) return;
        const int64_t warp = (blockIdx.x - s.tiles) * (kThreads / 32) + (threadIdx.x >> 5);
        zero_unsorted_rows<TO, VEC>(a, m, warp * 32, [&](int64_t p) { return key_at(s, m, p); });
        return;
    }
    const uint2* sorted = reinterpret_cast<const uint2*>(s.sorted.entries) + m * n;
    const int64_t col0 = (int64_t)blockIdx.y * s.columns;
    const int64_t p0 = blockIdx.x * s.tile;
    const uint2 kt = threadIdx.x < s.tile && p0 + threadIdx.x < n ? sorted[p0 + threadIdx.x] : make_uint2(kNone, 0u);
    pairs[threadIdx.x] = kt;
    const int count = __syncthreads_count(kt.x != kNone);
    if (count == 0) return;
    float* part = s.part + ((int64_t)m * s.tiles + blockIdx.x) * 2 * a.width;
    Around around;
    around.before = p0 > 0 && sorted[p0 - 1].x == pairs[0].x;
    around.after = p0 + count < n && sorted[p0 + count].x == pairs[count - 1].x;
    around.head = part;
    around.tail = part + a.width;
    sum_list<TO, VEC, Terms, kThreads>(
        a, m, TermsOf{a, m}, [&](int p) { return pairs[p]; }, [](uint32_t v) { return v; }, count, s.log2L, col0,
        reinterpret_cast<float*>(heads), around, [] { __syncthreads(); });
}

// Adds the sums of the runs that begin in a tile and go on in the next ones.  A warp
// has a tile and 32 vectors of columns (blockIdx.y); runs of many tiles are added by
// all of the CTA's warps, every 8th tile each, and the warps' sums in order.
constexpr int kLongRun = 16;

template <typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SumArgs s) {
    constexpr int kWarps = kThreads / 32;
    using P = Pack<float, VEC>;
    after_previous();
    const RowSumArgs& a = s.a;
    const int m = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = a.index.n;
    const int64_t tile = blockIdx.x * (int64_t)kWarps + warp;
    const int64_t p0 = tile * s.tile, p1 = p0 + s.tile;
    const int64_t col = ((int64_t)blockIdx.y * 32 + lane) * VEC;
    const float* part = s.part + (int64_t)m * s.tiles * 2 * a.width + col;
    __shared__ uint32_t long_key[kWarps];
    __shared__ int64_t long_last[kWarps];
    __shared__ P sums[kWarps][32];
    uint32_t key = kNone;
    int64_t last = tile + 1;    // the last tile whose first token is of the run
    if (p1 < n) {
        const uint32_t next = key_at(s, m, p1), end = key_at(s, m, p1 - 1);
        const uint32_t before = p0 > 0 ? key_at(s, m, p0 - 1) : kNone;
        if (end == next && end != before) key = end;
    }
    if (key != kNone) {
        auto has = [&](int64_t t) { return t < s.tiles && key_at(s, m, t * s.tile) == key; };
        int64_t step = 1;
        while (has(last + step)) {
            last += step;
            step *= 2;
        }
        for (; step > 0; step >>= 1)
            if (has(last + step)) last += step;
    }
    const bool is_long = key != kNone && last - tile > kLongRun;
    if (lane == 0) {
        long_key[warp] = is_long ? key : kNone;
        long_last[warp] = last;
    }
    P acc;
    auto add = [&](const float* src) {
        const P x = *reinterpret_cast<const P*>(src);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc.v[e] += x.v[e];
    };
    if (key != kNone && !is_long && col < a.width) {
        acc = *reinterpret_cast<const P*>(part + (tile * 2 + 1) * a.width);
#pragma unroll 4
        for (int64_t t = tile + 1; t <= last; ++t) add(part + t * 2 * a.width);
        write_row<TO, VEC>(a, m, key, col, acc.v);
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        if (long_key[w] == kNone) continue;
        const int64_t t0 = blockIdx.x * (int64_t)kWarps + w;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc.v[e] = 0.f;
        if (col < a.width) {
            if (warp == 0) add(part + (t0 * 2 + 1) * a.width);
#pragma unroll 4
            for (int64_t t = t0 + 1 + warp; t <= long_last[w]; t += kWarps) add(part + t * 2 * a.width);
        }
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp == 0 && col < a.width) {
            for (int k = 1; k < kWarps; ++k) add(sums[k][lane].v);
            write_row<TO, VEC>(a, m, long_key[w], col, acc.v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host

inline int64_t most_rows(const IndexArgs& x) {
    int64_t rows = 0;
    for (int m = 0; m < x.d; ++m) rows = x.rows[m] > rows ? x.rows[m] : rows;
    return rows;
}

// The rows' distribution over the CTAs of own_kernel for rows in vectors of `vec`
// elements; false where there are too many tokens or rows for it.
inline bool plan_own(const IndexArgs& index, int64_t width, int out_type, int vec, OwnArgs& o, dim3& grid) {
    if (index.n > kOwnTokens) return false;
    const int64_t rows = most_rows(index);
    // A row by as many lanes as it has vectors, in one part; with more tokens in parts of a
    // warp or 128 columns, so that a frequent row's are shared by more CTAs (16384 tokens, u^3
    // over 1024 rows of 1024 bf16: 35 us, against 69 us in one part; 4034 fp32 columns at odd
    // offsets, 12000 tokens over 2048 rows: 117 us by a warp, 93 in parts of 128 columns, 76
    // of 256, but 16000 u^3 over 200 rows of 513: 39, 52 and 78; 48 tokens over 512 rows of
    // 256: 6.0 us in two parts, 5.5 us in one).
    int most = index.n < 1024 ? 9 : 5;
    while ((vec << most) < 128) ++most;
    o.log2L = 0;
    while (o.log2L < most && ((int64_t)vec << o.log2L) < width) ++o.log2L;
    o.part = (int64_t)vec << o.log2L;
    const int64_t parts = cdiv(width, o.part);
    int64_t owners = kSms / (parts * index.d);
    owners = owners < 1 ? 1 : owners;
    // neighbouring rows stay together up to 1 KB, as long as every CTA gets eight blocks of them
    o.row_shift = 0;
    const int64_t row_bytes = width * elem_bytes(out_type);
    while ((row_bytes << o.row_shift) < 1024 && (rows >> (o.row_shift + 1)) >= 8 * owners) ++o.row_shift;
    const int64_t blocks = cdiv(rows, (int64_t)1 << o.row_shift);
    owners = owners < blocks ? owners : blocks;
    const int64_t owned = cdiv(blocks, owners) << o.row_shift;
    if (owned > kOwnRows || parts > 65535) return false;
    o.owned = (uint32_t)owned;
    o.per_warp = (uint32_t)(cdiv(index.n, kOwnThreads) * 32);
    grid = dim3((unsigned)owners, (unsigned)parts, index.d);
    return true;
}

// bytes of the partial sums, two rows for every tile
inline size_t part_bytes(const IndexArgs& x, int64_t width) {
    return sizeof(float) * x.d * cdiv(x.n, tile_tokens(x.n)) * 2 * width;
}

// Zeros of more than this many bytes are worth a launch in which the SMs share them as
// they get free, for few tokens too.  (4000 tokens into fp32 rows of 256 columns, by
// own_kernel and so: 64 MB 15 and 26 us, 96 MB 20 and 29, 128 MB 25 and 29, 192 MB 36 and
// 35, 400 MB 69 and 63; 16384 tokens: 96 MB 24 and 32, 128 MB 31 and 33, 192 MB 41 and 38;
// 4000 tokens, 33 columns: 96 MB 25 and 31, 128 MB 32 and 32, 192 MB 72 and 36.)
constexpr int64_t kFillBytes = 128 << 20;

// whether own_kernel takes the sums whatever the alignment of the rows (one launch that
// needs no workspace)
inline bool always_owned(const IndexArgs& index, int64_t width) {
    OwnArgs o;
    dim3 grid;
    bool all = index.d > 1 || index.rows[0] * width * 4 <= kFillBytes;
    for (int type : {MTTKRP_F32, MTTKRP_F16})
        for (int vec : {1, 2, 4, 8}) all = all && plan_own(index, width, type, vec, o, grid);
    return all;
}

// joins the tiles' crossing runs
template <typename TO, int VEC>
cudaError_t join(const SumArgs& s, cudaStream_t st) {
    if (s.tiles < 2) return cudaSuccess;
    const dim3 grid((unsigned)cdiv(s.tiles, kThreads / 32), (unsigned)cdiv(s.a.width, 32 * VEC), s.a.index.d);
    return launch_early(join_kernel<TO, VEC>, grid, kThreads, 0, st, s);
}

// Few: the terms as own_kernel takes them, whose CTAs of 1024 threads have few
// registers a thread; Many: as row_sum_kernel takes them; with kFewRing and kManyRing
// bytes of dynamic shared memory a thread that adds
template <typename TO, int VEC, template <typename> typename Few, int kFewRing, template <typename> typename Many,
          int kManyRing>
cudaError_t sums_by(const RowSumArgs& a, cudaStream_t st) {
    OwnArgs o;
    dim3 grid;
    const int64_t bytes = a.index.rows[0] * a.width * (int64_t)sizeof(TO);
    const bool fill = !a.accumulate && a.index.d == 1 && a.index.n > 0 && a.index.n <= kOwnTokens &&
                      a.out_stride == a.width && reinterpret_cast<uintptr_t>(a.out[0]) % 16 == 0 && bytes > kFillBytes;
    if (!fill && plan_own(a.index, a.width, a.out_type, VEC, o, grid)) {
        o.a = a;
        const size_t list = sizeof(uint32_t) * kOwnWarps * o.per_warp;
        o.first_bytes = (uint32_t)align256(list > kFewRing * kSumThreads ? list : kFewRing * kSumThreads);
        const size_t smem = o.first_bytes + sizeof(float) * kSumThreads * VEC +
                            sizeof(uint32_t) * (o.owned + (o.owned + 31) / 32) + list;
        constexpr auto kernel = own_kernel<TO, VEC, Few>;
        cudaError_t e = allow_smem<kernel>();
        if (e != cudaSuccess) return e;
        return launch_early(kernel, grid, kOwnThreads, smem, st, o);
    }
    const SortPlan p = plan_sort(a.index, sizeof(uint2), sort_sms());
    SumArgs s;
    s.a = a;
    s.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + p.total());
    s.tile = tile_tokens(a.index.n);
    s.tiles = cdiv(a.index.n, s.tile);
    s.log2L = 0;
    while ((1 << s.log2L) < kThreads && ((int64_t)VEC << s.log2L) < a.width) ++s.log2L;
    s.columns = (int64_t)VEC << s.log2L;
    cudaError_t e = fill ? sort_and_fill(a.index, p, a.ws, a.out[0], bytes, s.sorted, st)
                         : sort_tokens(a.index, p, a.ws, nullptr, nullptr, s.sorted, st);
    const int64_t zeros = a.accumulate || fill ? 0 : cdiv(most_rows(a.index), kThreads);
    if (e != cudaSuccess || s.tiles + zeros == 0) return e;
    constexpr auto kernel = row_sum_kernel<TO, VEC, Many>;
    e = allow_smem<kernel>();
    if (e != cudaSuccess) return e;
    const dim3 sum_grid((unsigned)(s.tiles + zeros), (unsigned)cdiv(a.width, s.columns), a.index.d);
    e = launch_early(kernel, sum_grid, kThreads, kThreads * kManyRing, st, s);
    if (e != cudaSuccess) return e;
    return join<TO, VEC>(s, st);
}

}  // namespace
}  // namespace mk
