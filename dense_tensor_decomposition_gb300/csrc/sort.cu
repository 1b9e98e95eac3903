// Sort of tokens by the row that they point to; see sort.h.
#include "rows.cuh"

namespace mk {
namespace {

// Stable radix sort of tokens by the row that they point to.  A pass of `bits` bits takes two
// launches over `ctas` CTAs for each index column, each with `per_cta` consecutive
// pairs: one counts the digits, one adds up the counts before its own and places its
// pairs, kSortTile at a time.  Tokens that take no part have row kNone, whose digits
// are all ones, and end up last.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 8;
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
    uint4* entries;         // the last pass's output as entries of 16 bytes, or nullptr
    const float* g;
    Tables tables[MTTKRP_MAX_ORDER];
};

// pair t of the pass's input
__device__ __forceinline__ uint2 sort_pair(const SortArgs& a, int64_t t, int m) {
    return a.src ? __ldcg(a.src + m * a.index.n + t) : make_uint2(sort_key(a.index, t, m), (uint32_t)t);
}

// the entry of 16 bytes for a token of column m
__device__ __forceinline__ uint4 entry_of(const SortArgs& a, uint2 kt, int m) {
    uint4 e = make_uint4(kt.x, 0u, 0u, 0u);
    if (kt.x == kNone) return e;
    e.y = __float_as_uint(a.g[kt.y]);
    uint32_t row[kMaxGroups] = {};
#pragma unroll
    for (int k = 0; k < kMaxGroups; ++k)
        if (k < a.tables[m].groups) row[k] = table_row(a.index, a.tables[m].group[k], kt.y);
    e.z = row[0] | row[1] << 16;
    e.w = row[2] | row[3] << 16;
    return e;
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
        if (a.entries) {
#pragma unroll
            for (int i = 0; i < kSortItems; ++i)
                if (digit[i] != kNone) a.entries[m * n + wh[digit[i]] + before[i]] = entry_of(a, kt[i], m);
        } else {
#pragma unroll
            for (int i = 0; i < kSortItems; ++i)
                if (digit[i] != kNone) __stcg(dst + wh[digit[i]] + before[i], kt[i]);
        }
    }
}

}  // namespace

SortPlan plan_sort(const IndexArgs& x, int entry_bytes) {
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
    p.pairs = align256((size_t)entry_bytes * x.d * x.n);
    p.counts = align256(sizeof(uint32_t) * x.d * p.ctas << p.bits);
    return p;
}

cudaError_t sort_tokens(const IndexArgs& index, const SortPlan& p, void* ws, const Tables* tables, const float* g,
                        Sorted& sorted, cudaStream_t s) {
    char* buf[2] = {static_cast<char*>(ws), static_cast<char*>(ws) + p.pairs};
    const size_t smem = sizeof(uint32_t) * (((kSortWarps + 1) << p.bits) + 2 * kSortThreads);
    cudaError_t e = allow_smem<sort_place_kernel>();
    if (e != cudaSuccess) return e;
    SortArgs a;
    a.index = index;
    a.src = nullptr;
    a.counts = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + 2 * p.pairs);
    a.bits = p.bits;
    a.per_cta = p.per_cta;
    a.entries = nullptr;
    a.g = g;
    if (tables)
        for (int m = 0; m < index.d; ++m) a.tables[m] = tables[m];
    const dim3 grid(p.ctas, index.d);
    for (int pass = 0; pass < p.passes; ++pass) {
        a.dst = reinterpret_cast<uint2*>(buf[pass & 1]);
        if (tables && pass == p.passes - 1) a.entries = reinterpret_cast<uint4*>(buf[pass & 1]);
        a.shift = pass * p.bits;
        sort_count_kernel<<<grid, kSortThreads, 0, s>>>(a);
        sort_place_kernel<<<grid, kSortThreads, smem, s>>>(a);
        a.src = a.dst;
    }
    sorted.entries = reinterpret_cast<const char*>(a.src);
    sorted.bytes = tables ? sizeof(uint4) : sizeof(uint2);
    return cudaGetLastError();
}

}  // namespace mk
