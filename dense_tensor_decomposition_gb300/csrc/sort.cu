// Sort of tokens by the row that they point to; see sort.h.
#include <cooperative_groups.h>

#include "rows.cuh"

namespace cg = cooperative_groups;

namespace mk {
namespace {

// Stable radix sort of tokens by the row that they point to: `ctas` CTAs for each index
// column, each with `per_cta` consecutive tokens, in one cooperative launch.  A pass of
// `bits` bits counts the digits (every warp those of its own consecutive tokens), waits
// for all CTAs, adds up the counts of smaller digits and of the CTAs before, and places
// the tokens.  With one tile a CTA the tokens and their ranks stay in registers between
// the two halves.  Tokens that take no part have row kNone and end up last: a single
// pass gives them the digit above the last row's, more passes see digits of all ones.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 10;

struct SortArgs {
    IndexArgs index;
    uint2* buf[2];          // d x n pairs each; pass k writes buf[k & 1]
    uint32_t* counts;       // d x ctas x bins
    int passes, bits;
    int bins;               // digits: 2^bits, or one more than the most rows in a single pass
    int64_t per_cta;
    char* entries;          // the last pass's output as entries of `entry_bytes` bytes, or nullptr
    int entry_bytes;
    const float* g;
    Tables tables[MTTKRP_MAX_ORDER];
};

// Writes the entries of 16 or 32 bytes of N tokens (row, token) of column m to entry
// numbers to[] (kNone: nowhere).  What it reads of the tokens' indices is used only where
// they take part.
template <int N>
__device__ __forceinline__ void write_entries(const SortArgs& a, const uint2* kt, const uint32_t* to, int m) {
    uint32_t g[N], rows[N][kMaxGroups / 2];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        g[u] = to[u] != kNone ? __float_as_uint(a.g[kt[u].y]) : 0u;
#pragma unroll
        for (int w = 0; w < kMaxGroups / 2; ++w) rows[u][w] = 0;
    }
    const int groups = a.tables[m].groups;
    for (int k = 0; k < groups; ++k) {
        const Tables::Group& group = a.tables[m].group[k];
        uint32_t row[N];
#pragma unroll
        for (int u = 0; u < N; ++u) row[u] = 0;
        for (int i = 0; i < group.modes; ++i) {
            const int mode = group.mode[i];
            const uint32_t size = (uint32_t)a.index.rows[mode];
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (to[u] != kNone) row[u] = row[u] * size + (uint32_t)index_at(a.index, kt[u].y, mode);
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t x = (group.first + row[u] & 0xFFFFu) << (k & 1) * 16;
#pragma unroll
            for (int w = 0; w < kMaxGroups / 2; ++w) rows[u][w] |= k / 2 == w ? x : 0u;
        }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (to[u] == kNone) continue;
        char* e = a.entries + ((int64_t)m * a.index.n + to[u]) * a.entry_bytes;
        *reinterpret_cast<uint4*>(e) = make_uint4(kt[u].x, g[u], rows[u][0], rows[u][1]);
        if (a.entry_bytes > 16) *reinterpret_cast<uint2*>(e + 16) = make_uint2(rows[u][2], rows[u][3]);
    }
}

// lanes of the warp with this lane's digit, which has at most `bits` bits or is kNone
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, int bits) {
    uint32_t peers = __ballot_sync(0xFFFFFFFFu, digit != kNone);
    for (int b = 0; b < bits; b += 2) {
        const bool one = (digit >> b & 1u) != 0, two = (digit >> b & 2u) != 0;
        const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one), twos = __ballot_sync(0xFFFFFFFFu, two);
        peers &= (one ? ones : ~ones) & (two ? twos : ~twos);
    }
    return peers;
}

// Column m by CTA `cta` of `ctas`, which wait(): wait for one another
template <int kSortItems, typename Wait>
__device__ __forceinline__ void sort_column(const SortArgs& a, int m, int cta, int ctas, const Wait& wait) {
    extern __shared__ uint32_t sort_smem[];
    constexpr int kSortTile = kSortThreads * kSortItems;
    const int nb = a.bins;
    uint32_t* whist = sort_smem;                    // kSortWarps x nb
    uint32_t* first = sort_smem + kSortWarps * nb;  // nb: counts of the CTA's digits, then their next places
    uint32_t* extra = first + nb;                   // 2 x kSortThreads
    __shared__ uint32_t sums[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n = a.index.n;
    const int64_t t0 = cta * a.per_cta;
    const int64_t t1 = t0 + a.per_cta < n ? t0 + a.per_cta : n;
    uint32_t* wh = whist + warp * nb;

    const bool one_tile = t0 + kSortTile >= t1;
    // a warp has kSortItems * 32 consecutive tokens of a tile
    uint2 kt[kSortItems];
    uint32_t place[kSortItems];     // digit, and << 16 how many of the warp's tokens with it come first; kNone: no token
    auto load_tile = [&](int pass, int64_t tile) {
        const uint2* src = a.buf[(pass + 1) & 1] + m * n;
        const int64_t w0 = tile + warp * (kSortItems * 32) + lane;
        if (pass == 0) {
            with_key(a.index, [&](auto key_of) {
#pragma unroll
                for (int i = 0; i < kSortItems; ++i) {
                    const int64_t t = w0 + i * 32;
                    kt[i] = make_uint2(t < t1 ? key_of(a.index, t, m) : kNone, (uint32_t)t);
                    if (i % 4 == 3) asm volatile("" ::: "memory");      // four tokens' loads at once: registers
                }
            });
        } else {
#pragma unroll
            for (int i = 0; i < kSortItems; ++i)
                kt[i] = w0 + i * 32 < t1 ? __ldcg(src + w0 + i * 32) : make_uint2(kNone, 0u);
        }
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            place[i] = kNone;
            if (w0 + i * 32 < t1)
                place[i] = a.passes == 1 ? min(kt[i].x, (uint32_t)nb - 1) : (kt[i].x >> pass * a.bits) & (nb - 1);
        }
    };
    auto rank_tile = [&]() {
        __syncthreads();            // what stood in whist has been read
        for (int i = tid; i < kSortWarps * nb; i += kSortThreads) whist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const uint32_t digit = place[i], peers = same_digit(digit, a.bits);
            const uint32_t rank = __popc(peers & ((1u << lane) - 1));
            if (digit != kNone) place[i] = digit | (wh[digit] + rank) << 16;
            __syncwarp();
            if (digit != kNone && rank == 0) wh[digit] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
    };

    for (int pass = 0; pass < a.passes; ++pass) {
        if (one_tile) {
            load_tile(pass, t0);
            rank_tile();
            for (int b = tid; b < nb; b += kSortThreads) {
                uint32_t c = 0;
#pragma unroll 8
                for (int w = 0; w < kSortWarps; ++w) c += whist[w * nb + b];
                first[b] = c;
            }
        } else {
            for (int b = tid; b < nb; b += kSortThreads) first[b] = 0;
            __syncthreads();
            for (int64_t tile = t0; tile < t1; tile += kSortTile) {
                load_tile(pass, tile);
#pragma unroll
                for (int i = 0; i < kSortItems; ++i)
                    if (place[i] != kNone) atomicAdd(first + place[i], 1u);
            }
            __syncthreads();
        }
        uint32_t* counts = a.counts + (int64_t)m * ctas * nb;
        for (int b = tid; b < nb; b += kSortThreads) __stcg(counts + cta * nb + b, first[b]);
        wait();
        // tokens with this digit in the CTAs before, and in all: every digit is added up
        // by kSortThreads / nb threads (nb <= kSortThreads)
        {
            const int splits = kSortThreads / nb, split = tid / nb, b = tid - split * nb;
            uint32_t less = 0, total = 0;
            if (split < splits) {
#pragma unroll 8
                for (int k = split; k < ctas; k += splits) {
                    const uint32_t x = __ldcg(counts + k * nb + b);
                    total += x;
                    less += k < cta ? x : 0;
                }
            }
            extra[tid] = less;
            extra[kSortThreads + tid] = total;
            __syncthreads();
            less = total = 0;
            if (tid < nb) {
                for (int k = 0; k < splits; ++k) {
                    less += extra[k * nb + b];
                    total += extra[kSortThreads + k * nb + b];
                }
            }
            uint32_t all;
            const uint32_t smaller = scan_warps<kSortWarps>(total, sums, all, [] { __syncthreads(); });
            if (tid < nb) first[b] = smaller + less;
        }
        uint2* dst = a.buf[pass & 1] + m * n;
        const bool last = pass == a.passes - 1;
        for (int64_t at = t0; at < t1; at += kSortTile) {
            if (!one_tile) {
                load_tile(pass, at);
                rank_tile();
            }
            __syncthreads();
            for (int b = tid; b < nb; b += kSortThreads) {
                uint32_t next = first[b];
                for (int w = 0; w < kSortWarps; w += 8) {
                    uint32_t c[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) c[k] = whist[(w + k) * nb + b];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        whist[(w + k) * nb + b] = next;
                        next += c[k];
                    }
                }
                first[b] = next;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSortItems; ++i)
                if (place[i] != kNone) place[i] = wh[place[i] & 0xFFFFu] + (place[i] >> 16);
            if (last && a.entries) {
                constexpr int kTogether = kSortItems < 4 ? kSortItems : 4;
#pragma unroll
                for (int i = 0; i < kSortItems; i += kTogether) write_entries<kTogether>(a, kt + i, place + i, m);
            } else {
#pragma unroll
                for (int i = 0; i < kSortItems; ++i)
                    if (place[i] != kNone) __stcg(dst + place[i], kt[i]);
            }
        }
        if (!last) wait();
    }
}

template <int kSortItems>
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const __grid_constant__ SortArgs a) {
    sort_column<kSortItems>(a, blockIdx.y, blockIdx.x, gridDim.x, [] { cg::this_grid().sync(); });
}

// Zeros for a large result while one cluster of CTAs sorts few tokens, a tile each.  The
// zeros are cut into many CTAs for the SMs to take as they get free: 537 MB take 72 us
// so, and 84 us in equal shares of the SMs, which do not all reach the memory equally fast.
constexpr int kFillCluster = 4;
constexpr int kFillVecs = 16 * kSortThreads;    // 16-byte vectors of a CTA

__global__ void __cluster_dims__(kFillCluster, 1, 1) __launch_bounds__(kSortThreads, 1)
    sort_and_fill_kernel(const __grid_constant__ SortArgs a, char* out, int64_t bytes) {
    after_previous();
    if (blockIdx.x < kFillCluster) {
        sort_column<4>(a, 0, blockIdx.x, kFillCluster, [] { cg::this_cluster().sync(); });
        return;
    }
    const int64_t vecs = bytes / 16, v0 = (int64_t)(blockIdx.x - kFillCluster) * kFillVecs + threadIdx.x;
    uint4* to = reinterpret_cast<uint4*>(out);
#pragma unroll
    for (int u = 0; u < kFillVecs / kSortThreads; ++u)
        if (v0 + u * kSortThreads < vecs) to[v0 + u * kSortThreads] = make_uint4(0u, 0u, 0u, 0u);
    if (blockIdx.x == kFillCluster && threadIdx.x < bytes % 16) out[vecs * 16 + threadIdx.x] = 0;
}

}  // namespace

int sort_sms() {
    static std::atomic<int> cached[64];     // by device; setting it twice is harmless
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64 && cached[dev] > 0) return cached[dev];
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return kSms;      // the launch will tell
    if (sms > kSms) sms = kSms;
    if (dev < 64) cached[dev] = sms;
    return sms;
}

SortPlan plan_sort(const IndexArgs& x, int entry_bytes, int sms) {
    SortPlan p;
    // digits cover the rows and, above them, one value for tokens that take no part
    int64_t most = 0;
    for (int m = 0; m < x.d; ++m) most = x.rows[m] > most ? x.rows[m] : most;
    int bits = 1;
    while (((int64_t)1 << bits) <= most) ++bits;
    p.passes = (int)cdiv(bits, kMaxDigit);
    p.bits = (int)cdiv(bits, p.passes);
    p.bins = p.passes == 1 ? (int)most + 1 : 1 << p.bits;
    // At most as many CTAs as are resident at once.  Tiles of 1024, 4096 or 8192 tokens: small
    // ones for the shortest way through a pass, until adding up the CTAs' counts takes longer
    // (20000 tokens in two passes: 19 us in tiles of 1024, 26 us in tiles of 4096; 524288: 29
    // us in tiles of 4096, 33 us in tiles of 8192).
    const int64_t n = x.n > 0 ? x.n : 1;
    const int64_t most_ctas = sms > x.d ? sms / x.d : 1;
    const int64_t few = most_ctas < 64 ? most_ctas : 64;
    p.items = n <= few * kSortThreads ? 1 : n <= most_ctas * kSortThreads * 4 ? 4 : 8;
    const int64_t tile = kSortThreads * p.items;
    p.per_cta = cdiv(cdiv(n, most_ctas), tile) * tile;
    p.ctas = (int)cdiv(n, p.per_cta);
    p.entry_bytes = entry_bytes;
    p.pairs = align256((size_t)entry_bytes * x.d * x.n);
    p.counts = align256(sizeof(uint32_t) * x.d * (p.ctas > kFillCluster ? p.ctas : kFillCluster) * p.bins);
    return p;
}

namespace {

size_t sort_smem_bytes(const SortPlan& p) { return sizeof(uint32_t) * ((kSortWarps + 1) * p.bins + 2 * kSortThreads); }

// buffers in the workspace; the last pass's output is what `sorted` tells
SortArgs sort_args(const IndexArgs& index, const SortPlan& p, void* ws, bool tables, Sorted& sorted) {
    SortArgs a;
    a.index = index;
    for (int k = 0; k < 2; ++k) a.buf[k] = reinterpret_cast<uint2*>(static_cast<char*>(ws) + k * p.pairs);
    a.counts = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + 2 * p.pairs);
    a.passes = p.passes;
    a.bits = p.bits;
    a.bins = p.bins;
    a.per_cta = p.per_cta;
    a.entries = tables ? reinterpret_cast<char*>(a.buf[(p.passes - 1) & 1]) : nullptr;
    a.entry_bytes = p.entry_bytes;
    a.g = nullptr;
    sorted.entries = static_cast<char*>(ws) + ((p.passes - 1) & 1) * p.pairs;
    sorted.bytes = p.entry_bytes;
    return a;
}

template <int kSortItems>
cudaError_t launch_sort(SortArgs& a, const SortPlan& p, cudaStream_t s) {
    constexpr auto kernel = sort_kernel<kSortItems>;
    cudaError_t e = allow_smem<kernel>();
    if (e != cudaSuccess) return e;
    void* args[] = {&a};
    e = cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(p.ctas, a.index.d), dim3(kSortThreads),
                                    args, sort_smem_bytes(p), s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace

cudaError_t sort_tokens(const IndexArgs& index, const SortPlan& p, void* ws, const Tables* tables, const float* g,
                        Sorted& sorted, cudaStream_t s) {
    SortArgs a = sort_args(index, p, ws, tables != nullptr, sorted);
    if (index.n == 0) return cudaSuccess;
    a.g = g;
    if (tables)
        for (int m = 0; m < index.d; ++m) a.tables[m] = tables[m];
    return p.items == 1 ? launch_sort<1>(a, p, s) : p.items == 4 ? launch_sort<4>(a, p, s) : launch_sort<8>(a, p, s);
}

cudaError_t sort_and_fill(const IndexArgs& index, const SortPlan& p, void* ws, void* out, int64_t bytes,
                          Sorted& sorted, cudaStream_t s) {
    SortArgs a = sort_args(index, p, ws, false, sorted);
    a.per_cta = kSortThreads * 4;
    if (index.n > kFillCluster * a.per_cta) return cudaErrorInvalidValue;
    cudaError_t e = allow_smem<sort_and_fill_kernel>();
    if (e != cudaSuccess) return e;
    const unsigned blocks = kFillCluster * (1 + (unsigned)cdiv(bytes, 16 * kFillVecs * kFillCluster));
    return launch_early(sort_and_fill_kernel, blocks, kSortThreads, sort_smem_bytes(p), s, a, static_cast<char*>(out),
                        bytes);
}

}  // namespace mk
