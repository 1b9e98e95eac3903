// Operators on rows of tables: lookup, its gradient by sorted tokens, entries of
// a CP model and their gradient.  The formulas are in rows.h.
//
// A gradient adds, for every row of a table, a term of each token that points to
// the row, in the order of the tokens, so that results repeat bit by bit.  Two ways:
//   * few tokens: one launch.  Every CTA owns some of the rows, finds the tokens
//     that point to them, groups them by row and writes its rows, zeros included.
//   * many tokens: the tokens are sorted by row (stable radix sort over the whole
//     GPU), and CTAs walk the sorted tokens in tiles of equal length, however long a
//     row's run of tokens is; runs that cross tile borders are joined by a last launch.
// Both add with sum_list(), which splits a list of sorted tokens over groups of
// lanes and joins the runs that cross the groups' borders.
#include <atomic>

#include "rows.h"
#include "types.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNone = 0xFFFFFFFFu;     // no index: above every table's last row

__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename IT>
__device__ __forceinline__ int64_t index_at(const IndexArgs& a, int64_t t, int m) {
    return (int64_t) static_cast<const IT*>(a.idx)[t * a.stride + m];
}

__device__ __forceinline__ int64_t index_at(const IndexArgs& a, int64_t t, int m) {
    return a.bytes == 8 ? index_at<int64_t>(a, t, m) : index_at<int32_t>(a, t, m);
}

// ---------------------------------------------------------------- lookup

// Bound by memory (the rows met, and the result).  L lanes take one part of one
// row: U vectors of VEC elements each, L vectors apart, all loaded before the first
// is stored.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(kThreads) lookup_kernel(LookupArgs a, int log2L) {
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x & ((1 << log2L) - 1);
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2L;
    if (t >= a.index.n) return;
    const int step = VEC << log2L;
    const int c0 = (int)blockIdx.y * U * step + lane * VEC;
    const int width = (int)a.width;
    const int64_t v = index_at(a.index, t, 0);
    const bool inside = v >= 0 && v < a.index.rows[0];
    P x[U];
    if (inside) {
        const T* src = static_cast<const T*>(a.table) + v * a.table_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * step < width) x[u] = *reinterpret_cast<const P*>(src + c0 + u * step);
    }
    T* dst = static_cast<T*>(a.out) + t * a.out_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (c0 + u * step >= width) break;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[u].v[e] = from_f32<T>(inside ? a.scale * to_f32(x[u].v[e]) : 0.f);
        *reinterpret_cast<P*>(dst + c0 + u * step) = x[u];
    }
}

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

// The terms of B tokens at VEC columns: rows of the gradient, or products of factor
// rows.  All loads are issued before the first term is used; every token must be one
// that takes part.
template <typename T, int VEC, int B, bool CP>
struct Terms;

template <typename T, int VEC, int B>
struct Terms<T, VEC, B, false> {
    Pack<T, VEC> x[B];
    __device__ __forceinline__ void load(const RowSumArgs& a, int, const uint32_t* tok, int64_t col) {
#pragma unroll
        for (int j = 0; j < B; ++j)
            x[j] = *reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(a.grad) +
                                                          (int64_t)tok[j] * a.grad_stride + col);
    }
    __device__ __forceinline__ float at(int j, int e) const { return to_f32(x[j].v[e]); }
};

template <typename T, int VEC, int B>
struct Terms<T, VEC, B, true> {
    float v[B][VEC];
    __device__ __forceinline__ void load(const RowSumArgs& a, int m, const uint32_t* tok, int64_t col) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const float g = a.g[tok[j]];
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[j][e] = g;
        }
        for (int l = 0; l < a.index.d; ++l) {
            if (l == m) continue;
            Pack<T, VEC> x[B];
#pragma unroll
            for (int j = 0; j < B; ++j)
                x[j] = *reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(a.factor[l]) +
                                                              index_at(a.index, tok[j], l) * a.width + col);
#pragma unroll
            for (int j = 0; j < B; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] *= to_f32(x[j].v[e]);
        }
    }
    __device__ __forceinline__ float at(int j, int e) const { return v[j][e]; }
};

// What lies around a list: whether its first run began before it, whether its last
// one goes on after it, and where such runs' sums go (indexed by column).
struct Around {
    bool before, after;
    float* head;
    float* tail;
};

// Adds the terms of a list of `count` >= 1 tokens sorted by row, list(p) = (row,
// token), over the columns from col0 on, and writes the finished rows.  A group of
// L = 2^log2L threads (of kN in all, which sync() makes wait for one another) walks
// count / groups consecutive tokens; a lane has VEC columns.  A run that crosses
// groups is finished by the group in which it began, from the other groups' parts
// in `heads` (kN * VEC floats), in the order of the groups.
template <typename T, typename TO, int VEC, int B, bool CP, int kN, typename List, typename Row, typename Sync>
__device__ __forceinline__ void sum_list(const RowSumArgs& a, int m, const List& list, const Row& row_of, int count,
                                         int log2L, int64_t col0, float* heads, const Around& around,
                                         const Sync& sync) {
    const int L = 1 << log2L, groups = kN >> log2L;
    const int group = threadIdx.x >> log2L, lane = threadIdx.x & (L - 1);
    const int64_t col = col0 + lane * VEC;
    const bool on = col < a.width;
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
    if (p0 < p1 && on) {
        cur = list(p0).x;
        bool began_before = p0 > 0 ? list(p0 - 1).x == cur : around.before;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
        for (int p = p0; p < p1; p += B) {
            uint32_t key[B], tok[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const uint2 kt = list(p + j < p1 ? p + j : p);
                key[j] = kt.x;
                tok[j] = kt.y;
            }
            Terms<T, VEC, B, CP> terms;
            terms.load(a, m, tok, col);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (p + j < p1) {
                    if (key[j] != cur) {
                        if (began_before) put(own_head);
                        else write_row<TO, VEC>(a, m, row_of(cur), col, acc);
                        began_before = false;
                        cur = key[j];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[e] += terms.at(j, e);
                }
            }
        }
        const bool goes_on = p1 < count ? list(p1).x == cur : around.after;
        if (began_before) put(own_head);
        else if (goes_on) open = true;
        else write_row<TO, VEC>(a, m, row_of(cur), col, acc);
    }
    sync();
    if (!on) return;
    if (open) {
        int g = group + 1;
        for (; g * share < count && list(g * share).x == cur; ++g) add(heads + ((size_t)(g << log2L) + lane) * VEC);
        if (g * share >= count && around.after && list(count - 1).x == cur) put(around.tail + col);
        else write_row<TO, VEC>(a, m, row_of(cur), col, acc);
    }
    if (group == 0 && around.before) {
        const uint32_t first = list(0).x;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = own_head[e];
        for (int g = 1; g * share < count && list(g * share).x == first; ++g)
            add(heads + ((size_t)(g << log2L) + lane) * VEC);
        put(around.head + col);
    }
}

// Zeros for those of `rows` local rows, from local row r0 on, that no token points
// to, by one warp; row_of gives a local row's number in the table (kNone: none).
template <typename TO, int VEC, typename Touched, typename Row>
__device__ __forceinline__ void zero_rows(const RowSumArgs& a, int m, uint32_t r0, uint32_t rows, int64_t col0,
                                          uint32_t vecs, const Touched& touched, const Row& row_of) {
    Pack<TO, VEC> zero;
#pragma unroll
    for (int e = 0; e < VEC; ++e) zero.v[e] = from_f32<TO>(0.f);
    for (uint32_t i = threadIdx.x & 31; i < rows * vecs; i += 32) {
        const uint32_t r = i / vecs, c = i - r * vecs;
        if (touched(r0 + r)) continue;
        const uint32_t v = row_of(r0 + r);
        if (v == kNone) continue;
        *reinterpret_cast<Pack<TO, VEC>*>(static_cast<TO*>(a.out[m]) + (int64_t)v * a.out_stride + col0 +
                                          (int64_t)c * VEC) = zero;
    }
}

// the row that token t points to in column m, kNone where it takes no part
__device__ __forceinline__ uint32_t sort_key(const IndexArgs& a, int64_t t, int m) {
    uint32_t key = kNone;
    bool inside = true;
    for (int l = 0; l < a.d; ++l) {
        const int64_t v = index_at(a, t, l);
        inside = inside && v >= 0 && v < a.rows[l];
        if (l == m) key = (uint32_t)v;
    }
    return inside ? key : kNone;
}

// sum of x over the threads before this one, and over all (in `all`); sums: one
// word a warp, and the threads wait twice
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sums, uint32_t& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t scan = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += up;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    const uint32_t w = sums[lane];      // 32 warps
    uint32_t wscan = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, wscan, o);
        if (lane >= o) wscan += up;
    }
    all = __shfl_sync(0xFFFFFFFFu, wscan, 31);
    const uint32_t before = __shfl_sync(0xFFFFFFFFu, wscan - w, warp);
    return before + scan - x;
}

// ---------------------------------------------------------------- few tokens: one launch

constexpr int kOwnThreads = 1024;
constexpr int kOwnWarps = kOwnThreads / 32;
constexpr int kSumThreads = 512;        // of which these add, while the others write zeros
constexpr int kTokenBits = 14;
constexpr int kOwnTokens = 1 << kTokenBits;
constexpr int kOwnRows = 1 << 13;       // rows of a CTA

// Owners: blocks of 2^row_shift consecutive rows go to the CTAs (blockIdx.x) in turn,
// so that frequent rows, which often have small numbers, are spread.
struct OwnArgs {
    RowSumArgs a;
    int row_shift;
    uint32_t owned;         // most rows a CTA owns
    uint32_t per_warp;      // tokens a warp looks at
    int log2L;
    int64_t part;           // columns of a CTA (blockIdx.y)
};

template <typename T, typename TO, int VEC, int B, bool CP>
__global__ void __launch_bounds__(kOwnThreads, 1) own_kernel(const __grid_constant__ OwnArgs o) {
    extern __shared__ float4 own_smem[];
    const RowSumArgs& a = o.a;
    float* heads = reinterpret_cast<float*>(own_smem);                          // kSumThreads * VEC
    uint32_t* cursor = reinterpret_cast<uint32_t*>(heads + kSumThreads * VEC);  // owned: tokens of each row, then their places
    uint32_t* touched = cursor + o.owned;                                       // a bit for each owned row
    uint32_t* found = touched + (o.owned + 31) / 32;                            // tokens of the CTA's rows, a part a warp
    uint32_t* list = found + kOwnWarps * o.per_warp;                            // the same without gaps, then sorted
    __shared__ uint32_t warp_found[kOwnWarps], sums[kOwnWarps], next_unit;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.z;
    const uint32_t G = gridDim.x, n = (uint32_t)a.index.n, rows = (uint32_t)a.index.rows[m];
    const uint32_t low = (1u << o.row_shift) - 1;
    auto row_of = [&](uint32_t r) -> uint32_t {
        const uint64_t v = (((uint64_t)(r >> o.row_shift) * G + blockIdx.x) << o.row_shift) | (r & low);
        return v < rows ? (uint32_t)v : kNone;
    };

    // the CTA's tokens, as (owned row, token), in order in every warp's part
    for (uint32_t i = threadIdx.x; i < o.owned; i += kOwnThreads) cursor[i] = 0;
    if (threadIdx.x == 0) next_unit = 0;
    __syncthreads();
    uint32_t count = 0;
    for (uint32_t k = 0; k < o.per_warp; k += 32) {
        const uint32_t t = warp * o.per_warp + k + lane;
        const uint32_t v = t < n ? sort_key(a.index, t, m) : kNone;
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
    if (lane == 0) warp_found[warp] = count;
    __syncthreads();
    // gaps out; the counts become the rows' first places
    uint32_t total = 0, base = 0;
    for (int w = 0; w < kOwnWarps; ++w) {
        const uint32_t c = warp_found[w];
        base += w < warp ? c : 0;
        total += c;
    }
    for (uint32_t k = lane; k < count; k += 32) list[base + k] = found[warp * o.per_warp + k];
    const uint32_t per = (o.owned + kOwnThreads - 1) / kOwnThreads;
    uint32_t mine = 0, all;
    for (uint32_t k = 0; k < per; ++k) {
        const uint32_t r = threadIdx.x * per + k;
        mine += r < o.owned ? cursor[r] : 0;
    }
    uint32_t at = block_scan(mine, sums, all);
    for (uint32_t r = threadIdx.x; r < (o.owned + 31) / 32 * 32; r += kOwnThreads) {
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, r < o.owned && cursor[r] != 0);
        if (lane == 0) touched[r / 32] = bits;
    }
    __syncthreads();
    for (uint32_t k = 0; k < per; ++k) {
        const uint32_t r = threadIdx.x * per + k;
        if (r >= o.owned) break;
        const uint32_t c = cursor[r];
        cursor[r] = at;
        at += c;
    }
    __syncthreads();

    const int64_t col0 = (int64_t)blockIdx.y * o.part;
    if (warp < kSumThreads / 32 && total > 0) {
        auto sync = [] { asm volatile("barrier.sync 1, %0;" ::"n"(kSumThreads) : "memory"); };
        // in order of the tokens within each row: one warp places them 32 at a time
        if (warp == 0) {
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
        sync();
        auto at_place = [&](int p) { return make_uint2(found[p] >> kTokenBits, found[p] & (kOwnTokens - 1)); };
        sum_list<T, TO, VEC, B, CP, kSumThreads>(a, m, at_place, row_of, (int)total, o.log2L, col0, heads,
                                                 Around{false, false, nullptr, nullptr}, sync);
    }
    if (a.accumulate) return;
    const uint32_t vecs = (uint32_t)((a.width - col0 < o.part ? a.width - col0 : o.part) / VEC);
    const uint32_t unit = vecs >= 1024 ? 1 : 1024 / vecs;
    auto is_touched = [&](uint32_t r) { return r >= o.owned || (touched[r >> 5] >> (r & 31) & 1u) != 0; };
    for (;;) {
        uint32_t u = 0;
        if (lane == 0) u = atomicAdd(&next_unit, 1u);
        u = __shfl_sync(0xFFFFFFFFu, u, 0);
        if ((uint64_t)u * unit >= o.owned) break;
        zero_rows<TO, VEC>(a, m, u * unit, unit, col0, vecs, is_touched, row_of);
    }
}

// ---------------------------------------------------------------- many tokens: sort

// Stable radix sort of (row, token) pairs by row.  A pass of `bits` bits takes two
// launches over `ctas` CTAs for each index column, each with `per_cta` consecutive
// pairs: one counts the digits, one adds up the counts before its own and places its
// pairs, kSortTile at a time.  Tokens that take no part have row kNone, whose digits
// are all ones, and end up last.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 4;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxDigit = 10;
constexpr int kSortCtas = 128;

struct SortArgs {
    IndexArgs index;
    const uint2* src;       // d x n pairs; nullptr: the indices
    uint2* dst;
    uint32_t* counts;       // d x ctas x 2^bits
    int shift, bits;
    int64_t per_cta;
};

// pair t of the pass's input
__device__ __forceinline__ uint2 sort_pair(const SortArgs& a, int64_t t, int m) {
    return a.src ? __ldcg(a.src + m * a.index.n + t) : make_uint2(sort_key(a.index, t, m), (uint32_t)t);
}

__global__ void __launch_bounds__(kSortThreads, 1) sort_count_kernel(const __grid_constant__ SortArgs a) {
    __shared__ uint32_t hist[1 << kMaxDigit];
    const int nb = 1 << a.bits, m = blockIdx.y, lane = threadIdx.x & 31;
    for (int b = threadIdx.x; b < nb; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    const int64_t t0 = blockIdx.x * a.per_cta;
    const int64_t t1 = t0 + a.per_cta < a.index.n ? t0 + a.per_cta : a.index.n;
    for (int64_t base = t0 + (threadIdx.x & ~31); base < t1; base += kSortTile) {
        uint32_t digit[kSortItems];
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t t = base + i * kSortThreads + lane;
            digit[i] = t < t1 ? (sort_pair(a, t, m).x >> a.shift) & (nb - 1) : kNone;
        }
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit[i]);
            if (digit[i] != kNone && lane == __ffs(peers) - 1) atomicAdd(hist + digit[i], (uint32_t)__popc(peers));
        }
    }
    __syncthreads();
    uint32_t* out = a.counts + ((int64_t)m * gridDim.x + blockIdx.x) * nb;
    for (int b = threadIdx.x; b < nb; b += kSortThreads) out[b] = hist[b];
}

__global__ void __launch_bounds__(kSortThreads, 1) sort_place_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ uint32_t sort_smem[];
    const int nb = 1 << a.bits, m = blockIdx.y;
    uint32_t* whist = sort_smem;                    // kSortWarps x nb
    uint32_t* first = sort_smem + kSortWarps * nb;  // nb: next place of each digit
    uint32_t* extra = first + nb;                   // 2 x kSortThreads
    __shared__ uint32_t sums[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // pairs with this digit in the CTAs before, and in all: every digit is added up by
    // kSortThreads / nb threads
    {
        const int digit = threadIdx.x & (nb - 1), split = threadIdx.x >> a.bits, splits = kSortThreads >> a.bits;
        const uint32_t* c = a.counts + (int64_t)m * gridDim.x * nb + digit;
        uint32_t before = 0, total = 0;
#pragma unroll 8
        for (int k = split; k < (int)gridDim.x; k += splits) {
            const uint32_t x = __ldcg(c + (int64_t)k * nb);
            total += x;
            before += k < (int)blockIdx.x ? x : 0;
        }
        extra[threadIdx.x] = before;
        extra[kSortThreads + threadIdx.x] = total;
        __syncthreads();
        before = total = 0;
        if ((int)threadIdx.x < nb) {
            for (int k = 0; k < splits; ++k) {
                before += extra[k * nb + digit];
                total += extra[kSortThreads + k * nb + digit];
            }
        }
        uint32_t all;
        const uint32_t smaller = block_scan(total, sums, all);
        if ((int)threadIdx.x < nb) first[digit] = smaller + before;
    }
    const int64_t n = a.index.n;
    const int64_t t0 = blockIdx.x * a.per_cta;
    const int64_t t1 = t0 + a.per_cta < n ? t0 + a.per_cta : n;
    uint2* dst = a.dst + m * n;
    uint32_t* wh = whist + warp * nb;
    for (int64_t tile = t0; tile < t1; tile += kSortTile) {
        // a warp has kSortItems * 32 consecutive pairs of the tile
        uint2 kt[kSortItems];
        uint32_t digit[kSortItems];
        const int64_t w0 = tile + warp * (kSortItems * 32) + lane;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t t = w0 + i * 32;
            kt[i] = t < t1 ? sort_pair(a, t, m) : make_uint2(kNone, 0u);
            digit[i] = t < t1 ? (kt[i].x >> a.shift) & (nb - 1) : kNone;
        }
        __syncthreads();        // the places of the tile before are taken
        for (int i = threadIdx.x; i < kSortWarps * nb; i += kSortThreads) whist[i] = 0;
        __syncthreads();
        uint32_t before[kSortItems];    // pairs of the warp with the same digit that come first
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit[i]);
            const uint32_t rank = __popc(peers & ((1u << lane) - 1));
            before[i] = 0;
            if (digit[i] != kNone) before[i] = wh[digit[i]] + rank;
            __syncwarp();
            if (digit[i] != kNone && rank == 0) wh[digit[i]] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        for (int b = threadIdx.x; b < nb; b += kSortThreads) {
            uint32_t at = first[b];
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = whist[w * nb + b];
                whist[w * nb + b] = at;
                at += c;
            }
            first[b] = at;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i)
            if (digit[i] != kNone) __stcg(dst + wh[digit[i]] + before[i], kt[i]);
    }
}

// ---------------------------------------------------------------- many tokens: sums

constexpr int kTile = 256;              // sorted tokens of a CTA

struct SumArgs {
    RowSumArgs a;
    const uint2* sorted;    // d x n (row, token)
    float* part;            // d x tiles x 2 x width: sums of the tile's first run that began before, of its last that goes on
    int64_t tiles;
    int64_t zero_ctas;      // CTAs (blockIdx.x) behind the tiles' that write zeros
    int log2L;
    int64_t columns;        // columns of a CTA (blockIdx.y)
};

template <typename T, typename TO, int VEC, int B, bool CP>
__global__ void __launch_bounds__(kThreads) row_sum_kernel(const __grid_constant__ SumArgs s) {
    __shared__ uint2 pairs[kTile];
    __shared__ float4 heads[kThreads * VEC / 4 > 0 ? (kThreads * VEC + 3) / 4 : 1];
    const RowSumArgs& a = s.a;
    const int m = blockIdx.z;
    const int64_t n = a.index.n;
    const uint2* sorted = s.sorted + m * n;
    const int64_t col0 = (int64_t)blockIdx.y * s.columns;
    if (blockIdx.x >= s.tiles) {
        // 32 rows a warp; a lane looks one row up among the sorted tokens
        const int64_t r0 = ((blockIdx.x - s.tiles) * (kThreads / 32) + (threadIdx.x >> 5)) * 32;
        const int64_t rows = a.index.rows[m];
        if (r0 >= rows) return;
        const int64_t v = r0 + (threadIdx.x & 31);
        int64_t lo = 0, hi = n;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (__ldg(&sorted[mid].x) < v) lo = mid + 1;
            else hi = mid;
        }
        const bool has = v >= rows || (lo < n && sorted[lo].x == (uint32_t)v);
        const uint32_t touched = __ballot_sync(0xFFFFFFFFu, has);
        const uint32_t vecs = (uint32_t)((a.width - col0 < s.columns ? a.width - col0 : s.columns) / VEC);
        zero_rows<TO, VEC>(
            a, m, 0, 32, col0, vecs, [&](uint32_t r) { return (touched >> r & 1u) != 0; },
            [&](uint32_t r) { return (uint32_t)(r0 + r); });
        return;
    }
    const int64_t p0 = blockIdx.x * (int64_t)kTile;
    int count = 0;
#pragma unroll
    for (int i = 0; i < kTile; i += kThreads) {
        const int64_t p = p0 + i + threadIdx.x;
        const uint2 kt = p < n ? sorted[p] : make_uint2(kNone, 0u);
        pairs[i + threadIdx.x] = kt;
        count += __syncthreads_count(kt.x != kNone);
    }
    if (count == 0) return;
    float* part = s.part + ((int64_t)m * s.tiles + blockIdx.x) * 2 * a.width;
    Around around;
    around.before = p0 > 0 && sorted[p0 - 1].x == pairs[0].x;
    around.after = p0 + count < n && sorted[p0 + count].x == pairs[count - 1].x;
    around.head = part;
    around.tail = part + a.width;
    sum_list<T, TO, VEC, B, CP, kThreads>(
        a, m, [&](int p) { return pairs[p]; }, [](uint32_t v) { return v; }, count, s.log2L, col0,
        reinterpret_cast<float*>(heads), around, [] { __syncthreads(); });
}

// Adds the sums of the run that begins in a tile and goes on in the next ones.  A
// warp has a tile and 32 columns; runs of many tiles are added by all of the CTA's
// warps, every 8th tile each, and the warps' sums in order.
constexpr int kLongRun = 32;

template <typename TO>
__global__ void __launch_bounds__(kThreads) row_join_kernel(const __grid_constant__ SumArgs s) {
    constexpr int kWarps = kThreads / 32;
    const RowSumArgs& a = s.a;
    const int m = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = a.index.n, tile = blockIdx.x * (int64_t)kWarps + warp;
    const uint2* sorted = s.sorted + m * n;
    const int64_t p0 = tile * kTile, p1 = p0 + kTile;
    const float* part = s.part + (int64_t)m * s.tiles * 2 * a.width;
    const int64_t col = (int64_t)blockIdx.y * 32 + lane;
    __shared__ uint32_t long_key[kWarps];
    __shared__ int64_t long_last[kWarps];
    __shared__ float sums[kWarps][32];
    uint32_t key = kNone;
    int64_t last = 0;           // the last tile whose first token is of the run
    if (p1 < n) {
        const uint32_t next = sorted[p1].x, end = sorted[p1 - 1].x, before = p0 > 0 ? sorted[p0 - 1].x : kNone;
        if (end == next && end != before) key = end;
    }
    if (key != kNone) {
        int64_t step = 1;
        last = tile + 1;
        while (last + step < s.tiles && sorted[(last + step) * kTile].x == key) {
            last += step;
            step *= 2;
        }
        for (; step > 0; step >>= 1)
            if (last + step < s.tiles && sorted[(last + step) * kTile].x == key) last += step;
    }
    const bool is_long = key != kNone && last - tile > kLongRun;
    if (lane == 0) {
        long_key[warp] = is_long ? key : kNone;
        long_last[warp] = last;
    }
    float acc = 0.f;
    if (key != kNone && !is_long && col < a.width) {
        acc = part[(tile * 2 + 1) * a.width + col];
#pragma unroll 4
        for (int64_t t = tile + 1; t <= last; ++t) acc += part[t * 2 * a.width + col];
        write_row<TO, 1>(a, m, key, col, &acc);
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        if (long_key[w] == kNone) continue;
        const int64_t t0 = blockIdx.x * (int64_t)kWarps + w;
        acc = 0.f;
        if (col < a.width) {
            if (warp == 0) acc = part[(t0 * 2 + 1) * a.width + col];
#pragma unroll 8
            for (int64_t t = t0 + 1 + warp; t <= long_last[w]; t += kWarps) acc += part[t * 2 * a.width + col];
        }
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp == 0 && col < a.width) {
            for (int k = 1; k < kWarps; ++k) acc += sums[k][lane];
            write_row<TO, 1>(a, m, long_key[w], col, &acc);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- entries

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) entries_kernel(EntriesArgs a, int log2L) {
    const int L = 1 << log2L;
    const int lane = threadIdx.x & (L - 1);
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2L;
    const bool any = t < a.index.n;
    bool inside = any;
    for (int l = 0; any && l < a.index.d; ++l) {
        const int64_t v = index_at(a.index, t, l);
        inside = inside && v >= 0 && v < a.index.rows[l];
    }
    float sum = 0.f;
    if (inside) {
        for (int64_t c = (int64_t)lane * VEC; c < a.width; c += (int64_t)VEC << log2L) {
            float v[VEC];
            for (int l = 0; l < a.index.d; ++l) {
                const Pack<T, VEC> x = *reinterpret_cast<const Pack<T, VEC>*>(
                    static_cast<const T*>(a.factor[l]) + index_at(a.index, t, l) * a.width + c);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = l == 0 ? to_f32(x.v[e]) : v[e] * to_f32(x.v[e]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += v[e];
        }
    }
    for (int o = L >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (any && lane == 0) a.out[t] = sum;
}

// ---------------------------------------------------------------- host

constexpr size_t elem_bytes(int type) { return type == MTTKRP_F32 ? 4 : 2; }

// rows of `width` elements, `stride` apart, can be read and written 16 bytes at a time
bool wide(const void* p, int64_t stride, int64_t width, int type) {
    const size_t e = elem_bytes(type);
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * e) % 16 == 0 && (width * e) % 16 == 0;
}

// lanes for a row of `items` loads: a power of two, at most a warp
int log2_lanes(int64_t items) {
    int l = 0;
    while (l < 5 && ((int64_t)1 << l) < items) ++l;
    return l;
}

template <typename T, int VEC, int U>
cudaError_t lookup_by(const LookupArgs& a, cudaStream_t s) {
    const int l = log2_lanes(cdiv(a.width, VEC));
    const dim3 grid((unsigned)cdiv(a.index.n << l, kThreads), (unsigned)cdiv(a.width, (int64_t)(VEC * U) << l));
    lookup_kernel<T, VEC, U><<<grid, kThreads, 0, s>>>(a, l);
    return cudaGetLastError();
}

// the widest vectors that the rows' starts and width allow
template <typename T>
cudaError_t lookup(const LookupArgs& a, cudaStream_t s) {
    constexpr int e = sizeof(T);
    const size_t all = reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.out) |
                       (a.table_stride * e) | (a.out_stride * e) | (a.width * e);
    if (all % 16 == 0) return lookup_by<T, 16 / e, 4>(a, s);
    if (all % 4 == 0) return lookup_by<T, 4 / e, 8>(a, s);
    if constexpr (e < 4) return lookup_by<T, 1, 16>(a, s);
    return cudaErrorInvalidValue;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr size_t kMaxSmem = 200 * 1024;

// lets a kernel have kMaxSmem bytes of dynamic shared memory on the current device
template <auto kernel>
cudaError_t allow_smem() {
    static std::atomic<uint64_t> done{0};       // a bit a device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1) != 0)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    return e;
}

constexpr int kSms = 152;

// The rows' distribution over the CTAs of own_kernel for rows of `width` elements
// in vectors of `vec`; false where there are too many tokens or rows for it.
bool plan_own(const RowSumArgs& a, int vec, OwnArgs& o, dim3& grid) {
    if (a.index.n > kOwnTokens) return false;
    int64_t rows = 0;
    for (int m = 0; m < a.index.d; ++m) rows = a.index.rows[m] > rows ? a.index.rows[m] : rows;
    o.a = a;
    o.log2L = 0;
    while ((1 << o.log2L) < kSumThreads && ((int64_t)vec << o.log2L) < a.width) ++o.log2L;
    o.part = (int64_t)vec << o.log2L;
    const int64_t parts = cdiv(a.width, o.part);
    int64_t owners = kSms / (parts * a.index.d);
    owners = owners < 1 ? 1 : owners;
    // neighbouring rows stay together up to 1 KB, as long as every CTA gets eight blocks of them
    o.row_shift = 0;
    const int64_t row_bytes = a.width * elem_bytes(a.out_type);
    while ((row_bytes << o.row_shift) < 1024 && (rows >> (o.row_shift + 1)) >= 8 * owners) ++o.row_shift;
    const int64_t blocks = cdiv(rows, (int64_t)1 << o.row_shift);
    owners = owners < blocks ? owners : blocks;
    const int64_t owned = cdiv(blocks, owners) << o.row_shift;
    if (owned > kOwnRows || parts > 65535) return false;
    o.owned = (uint32_t)owned;
    o.per_warp = (uint32_t)(cdiv(a.index.n, kOwnThreads) * 32);
    grid = dim3((unsigned)owners, (unsigned)parts, a.index.d);
    return true;
}

// what the sort needs of the workspace: two lists of pairs, the counts, the sums of
// runs that cross tiles
struct SortPlan {
    int passes, bits, ctas;
    int64_t per_cta, tiles;
    size_t pairs, counts, part;     // bytes
};

SortPlan plan_sort(const IndexArgs& x, int64_t width) {
    SortPlan p;
    // digits cover the rows and, above them, one value for tokens that take no part
    int64_t most = 0;
    for (int m = 0; m < x.d; ++m) most = x.rows[m] > most ? x.rows[m] : most;
    int bits = 1;
    while (((int64_t)1 << bits) <= most) ++bits;
    p.passes = (int)cdiv(bits, kMaxDigit);
    p.bits = (int)cdiv(bits, p.passes);
    const int64_t n = x.n > 0 ? x.n : 1;
    p.per_cta = cdiv(cdiv(n, kSortCtas), kSortTile) * kSortTile;
    p.ctas = (int)cdiv(n, p.per_cta);
    p.tiles = cdiv(x.n, kTile);
    p.pairs = align256(sizeof(uint2) * x.d * x.n);
    p.counts = align256(sizeof(uint32_t) * x.d * p.ctas << p.bits);
    p.part = sizeof(float) * x.d * p.tiles * 2 * width;
    return p;
}

// sorts the tokens of every index column; fills in where the sums find them
cudaError_t sort_tokens(const RowSumArgs& a, SumArgs& s, cudaStream_t st) {
    const SortPlan p = plan_sort(a.index, a.width);
    char* ws = static_cast<char*>(a.ws);
    uint2* buf[2] = {reinterpret_cast<uint2*>(ws), reinterpret_cast<uint2*>(ws + p.pairs)};
    const size_t smem = sizeof(uint32_t) * (((kSortWarps + 1) << p.bits) + 2 * kSortThreads);
    cudaError_t e = allow_smem<sort_place_kernel>();
    if (e != cudaSuccess) return e;
    SortArgs so;
    so.index = a.index;
    so.src = nullptr;
    so.counts = reinterpret_cast<uint32_t*>(ws + 2 * p.pairs);
    so.bits = p.bits;
    so.per_cta = p.per_cta;
    const dim3 grid(p.ctas, a.index.d);
    for (int pass = 0; pass < p.passes; ++pass) {
        so.dst = buf[pass & 1];
        so.shift = pass * p.bits;
        sort_count_kernel<<<grid, kSortThreads, 0, st>>>(so);
        sort_place_kernel<<<grid, kSortThreads, smem, st>>>(so);
        so.src = so.dst;
    }
    s.a = a;
    s.sorted = so.src;
    s.part = reinterpret_cast<float*>(ws + 2 * p.pairs + p.counts);
    s.tiles = p.tiles;
    return cudaGetLastError();
}

template <typename T, typename TO, int VEC, bool CP>
cudaError_t sums_by(const RowSumArgs& a, cudaStream_t st) {
    constexpr int kB = CP ? 4 : 8;
    OwnArgs o;
    dim3 grid;
    if (plan_own(a, VEC, o, grid)) {
        const size_t smem = sizeof(float) * kSumThreads * VEC +
                            sizeof(uint32_t) * (o.owned + (o.owned + 31) / 32 + 2 * kOwnWarps * o.per_warp);
        constexpr auto kernel = own_kernel<T, TO, VEC, 4, CP>;
        cudaError_t e = allow_smem<kernel>();
        if (e != cudaSuccess) return e;
        kernel<<<grid, kOwnThreads, smem, st>>>(o);
        return cudaGetLastError();
    }
    const int64_t n = a.index.n;
    const int d = a.index.d;
    SumArgs s;
    cudaError_t e = sort_tokens(a, s, st);
    if (e != cudaSuccess) return e;
    s.log2L = 0;
    while ((1 << s.log2L) < kThreads && ((int64_t)VEC << s.log2L) < a.width) ++s.log2L;
    s.columns = (int64_t)VEC << s.log2L;
    int64_t rows = 0;
    for (int m = 0; m < d; ++m) rows = a.index.rows[m] > rows ? a.index.rows[m] : rows;
    s.zero_ctas = a.accumulate ? 0 : cdiv(rows, kThreads);
    const dim3 sum_grid((unsigned)(s.tiles + s.zero_ctas), (unsigned)cdiv(a.width, s.columns), d);
    row_sum_kernel<T, TO, VEC, kB, CP><<<sum_grid, kThreads, 0, st>>>(s);
    if (n > kTile) {
        const dim3 join((unsigned)cdiv(s.tiles, kThreads / 32), (unsigned)cdiv(a.width, 32), d);
        row_join_kernel<TO><<<join, kThreads, 0, st>>>(s);
    }
    return cudaGetLastError();
}

// rows in 16-byte vectors of the source's type where all starts allow it
template <typename T, typename TO, bool CP>
cudaError_t sums(const RowSumArgs& a, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T);
    bool w = CP || wide(a.grad, a.grad_stride, a.width, a.type);
    for (int m = 0; m < a.index.d; ++m) {
        constexpr size_t bytes = kVec * sizeof(TO);
        w = w && reinterpret_cast<uintptr_t>(a.out[m]) % bytes == 0 && a.out_stride * sizeof(TO) % bytes == 0;
        if (CP) w = w && wide(a.factor[m], a.width, a.width, a.type);
    }
    return w ? sums_by<T, TO, kVec, CP>(a, st) : sums_by<T, TO, 1, CP>(a, st);
}

template <typename T>
cudaError_t entries(const EntriesArgs& a, int type, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    bool w = true;
    for (int m = 0; m < a.index.d; ++m) w = w && wide(a.factor[m], a.width, a.width, type);
    const int l = log2_lanes(w ? cdiv(a.width, kVec) : a.width);
    const unsigned blocks = (unsigned)cdiv(a.index.n << l, kThreads);
    if (w) entries_kernel<T, kVec><<<blocks, kThreads, 0, s>>>(a, l);
    else entries_kernel<T, 1><<<blocks, kThreads, 0, s>>>(a, l);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, int type, cudaStream_t s) {
    if (a.index.n == 0) return cudaSuccess;
    if (type == MTTKRP_F32) return lookup<float>(a, s);
    if (type == MTTKRP_BF16) return lookup<__nv_bfloat16>(a, s);
    return lookup<__half>(a, s);
}

size_t row_sum_workspace_bytes(const IndexArgs& index, int64_t width) {
    const SortPlan p = plan_sort(index, width);
    return 2 * p.pairs + p.counts + p.part;
}

cudaError_t launch_row_sum(const RowSumArgs& a, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if (a.model) {
        if (a.type == MTTKRP_F32) return sums<float, float, true>(a, s);
        if (a.type == MTTKRP_BF16) return sums<bf16, float, true>(a, s);
        return sums<__half, float, true>(a, s);
    }
    if (a.type == MTTKRP_F32) return sums<float, float, false>(a, s);
    if (a.type == MTTKRP_BF16)
        return a.out_type == MTTKRP_F32 ? sums<bf16, float, false>(a, s) : sums<bf16, bf16, false>(a, s);
    return a.out_type == MTTKRP_F32 ? sums<__half, float, false>(a, s) : sums<__half, __half, false>(a, s);
}

cudaError_t launch_entries(const EntriesArgs& a, int type, cudaStream_t s) {
    if (a.index.n == 0) return cudaSuccess;
    if (type == MTTKRP_F32) return entries<float>(a, type, s);
    if (type == MTTKRP_BF16) return entries<__nv_bfloat16>(a, type, s);
    return entries<__half>(a, type, s);
}

}  // namespace mk
