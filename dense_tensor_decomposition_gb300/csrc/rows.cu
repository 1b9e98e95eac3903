// Operators on rows of tables: lookup, its gradient by sorted tokens, entries of
// a CP model and their gradient.  The formulas are in rows.h.
//
// The gradients sort the tokens by index (stable, so the order of every sum is
// fixed), then walk the sorted tokens in chunks: a chunk adds the rows of each
// run of equal indices in registers and writes the finished runs; runs that cross
// chunk borders leave partial sums, which a last kernel adds in order.
#include <cooperative_groups.h>

#include "rows.h"
#include "types.cuh"

namespace cg = cooperative_groups;

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

// One row by L lanes; a lane takes vectors of VEC elements, L apart.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) lookup_kernel(LookupArgs a, int log2L) {
    const int lane = threadIdx.x & ((1 << log2L) - 1);
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2L;
    if (t >= a.index.n) return;
    const int64_t v = index_at(a.index, t, 0);
    const bool inside = v >= 0 && v < a.index.rows[0];
    const T* src = static_cast<const T*>(a.table) + (inside ? v : 0) * a.table_stride;
    T* dst = static_cast<T*>(a.out) + t * a.out_stride;
    for (int64_t c = (int64_t)lane * VEC; c < a.width; c += (int64_t)VEC << log2L) {
        Pack<T, VEC> x;
        if (inside) x = *reinterpret_cast<const Pack<T, VEC>*>(src + c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x.v[e] = from_f32<T>(inside ? a.scale * to_f32(x.v[e]) : 0.f);
        *reinterpret_cast<Pack<T, VEC>*>(dst + c) = x;
    }
}

// ---------------------------------------------------------------- sort

// Stable radix sort of (index, token) pairs by index, one cluster of kCluster
// CTAs for each of the d index columns.  A pass: every warp counts the digits of
// its own consecutive tokens; the CTAs exchange their counts through distributed
// shared memory; every warp then places its tokens in order.  Tokens that take
// no part get the index kNone's digits (all ones) and end up last.
constexpr int kCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 10;

struct SortArgs {
    IndexArgs index;
    uint2* buf[2];          // d x n pairs each
    int passes, bits;       // of `bits` bits each
    int first;              // buffer that the first pass writes; the last pass writes buf[1]
};

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

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads, 1) sort_kernel(SortArgs a) {
    extern __shared__ uint32_t sm[];
    const int nb = 1 << a.bits;
    uint32_t* whist = sm;                       // [kSortWarps][nb]
    uint32_t* count = sm + kSortWarps * nb;     // [nb], read by the other CTAs
    uint32_t* wsum = count + nb;                // [kSortWarps]
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int m = blockIdx.x / kCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = a.index.n;
    const int64_t per_warp = cdiv(cdiv(n, kCluster * kSortWarps), 32) * 32;
    const int64_t t0 = ((int64_t)rank * kSortWarps + warp) * per_warp;
    const int64_t t1 = t0 + per_warp < n ? t0 + per_warp : n;
    uint32_t* wh = whist + warp * nb;

    for (int pass = 0; pass < a.passes; ++pass) {
        const uint2* src = a.buf[(a.first + pass + 1) & 1] + m * n;
        uint2* dst = a.buf[(a.first + pass) & 1] + m * n;
        const int shift = pass * a.bits;
        const uint32_t mask = (uint32_t)nb - 1;
        for (int i = threadIdx.x; i < kSortWarps * nb; i += kSortThreads) whist[i] = 0;
        __syncthreads();
        for (int64_t base = t0; base < t1; base += 32) {
            const int64_t t = base + lane;
            uint32_t digit = kNone;             // a lane behind the last token: counted nowhere
            if (t < t1) digit = ((pass == 0 ? sort_key(a.index, t, m) : __ldcg(src + t).x) >> shift) & mask;
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
            if (t < t1 && lane == __ffs(peers) - 1) wh[digit] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        const int b = threadIdx.x;
        if (b < nb) {
            uint32_t c = 0;
            for (int w = 0; w < kSortWarps; ++w) c += whist[w * nb + b];
            count[b] = c;
        }
        cluster.sync();
        // first place of this CTA's digit b: all smaller digits, and digit b of the CTAs before
        uint32_t before = 0, total = 0;
        if (b < nb) {
            for (int r = 0; r < kCluster; ++r) {
                const uint32_t c = cluster.map_shared_rank(count, r)[b];
                total += c;
                if (r < rank) before += c;
            }
        }
        uint32_t scan = total;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
            if (lane >= o) scan += up;
        }
        if (lane == 31) wsum[warp] = scan;
        __syncthreads();
        if (b < nb) {
            uint32_t at = before + scan - total;
            for (int w = 0; w < warp; ++w) at += wsum[w];
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = whist[w * nb + b];
                whist[w * nb + b] = at;
                at += c;
            }
        }
        __syncthreads();
        for (int64_t base = t0; base < t1; base += 32) {
            const int64_t t = base + lane;
            uint2 kt = make_uint2(0u, 0u);
            uint32_t digit = kNone;
            if (t < t1) {
                kt = pass == 0 ? make_uint2(sort_key(a.index, t, m), (uint32_t)t) : __ldcg(src + t);
                digit = (kt.x >> shift) & mask;
            }
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
            uint32_t at = 0;
            if (t < t1) at = wh[digit] + __popc(peers & ((1u << lane) - 1));
            __syncwarp();
            if (t < t1 && lane == __ffs(peers) - 1) wh[digit] += __popc(peers);
            __syncwarp();
            if (t < t1) __stcg(dst + at, kt);
        }
        cluster.sync();
    }
}

// ---------------------------------------------------------------- sums of rows

struct SumArgs {
    RowSumArgs a;
    const uint2* sorted;    // d x n (index, token)
    float* part;            // d x chunks x 2 x width partial sums: [0] of a run that began before, [1] of one that goes on
    int chunk;              // tokens a chunk
    int64_t chunks;
    int log2L;              // lanes a row
};

template <typename TO, int VEC, int U>
__device__ __forceinline__ void write_row(const RowSumArgs& a, int m, uint32_t v, int64_t col, int step,
                                          const float* acc) {
    TO* dst = static_cast<TO*>(a.out[m]) + (int64_t)v * a.out_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = col + u * step;
        if (c >= a.width) continue;
        Pack<TO, VEC>* p = reinterpret_cast<Pack<TO, VEC>*>(dst + c);
        Pack<TO, VEC> x;
        if (a.accumulate) x = *p;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float s = a.scale * acc[u * VEC + e];
            x.v[e] = from_f32<TO>(a.accumulate ? to_f32(x.v[e]) + s : s);
        }
        *p = x;
    }
}

// the rows of tokens tok[0..B) into v (zeros where on[j] is false)
template <typename T, int VEC, int U, int B, bool CP>
__device__ __forceinline__ void load_rows(const RowSumArgs& a, int m, const uint32_t* tok, const bool* on,
                                          int64_t col, int step, float (*v)[U * VEC]) {
    using P = Pack<T, VEC>;
    if constexpr (!CP) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const T* src = static_cast<const T*>(a.grad) + (int64_t)tok[j] * a.grad_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = col + u * step;
                P x;
                const bool in = on[j] && c < a.width;
                if (in) x = *reinterpret_cast<const P*>(src + c);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][u * VEC + e] = in ? to_f32(x.v[e]) : 0.f;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const float gj = on[j] ? a.g[tok[j]] : 0.f;
#pragma unroll
            for (int e = 0; e < U * VEC; ++e) v[j][e] = gj;
        }
        for (int l = 0; l < a.index.d; ++l) {
            if (l == m) continue;
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int64_t row = on[j] ? index_at(a.index, tok[j], l) : 0;
                const T* src = static_cast<const T*>(a.factor[l]) + row * a.width;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = col + u * step;
                    P x;
                    const bool in = on[j] && c < a.width;
                    if (in) x = *reinterpret_cast<const P*>(src + c);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[j][u * VEC + e] *= in ? to_f32(x.v[e]) : 0.f;
                }
            }
        }
    }
}

// L lanes walk one chunk of the sorted tokens over L * U * VEC columns.
template <typename T, typename TO, int VEC, int U, int B, bool CP>
__global__ void __launch_bounds__(kThreads) row_sum_kernel(SumArgs s) {
    const RowSumArgs& a = s.a;
    const int L = 1 << s.log2L;
    const int lane = threadIdx.x & (L - 1);
    const int64_t chunk = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> s.log2L;
    if (chunk >= s.chunks) return;
    const int m = blockIdx.z;
    const int step = L * VEC;
    const int64_t col = (int64_t)blockIdx.y * step * U + lane * VEC;
    if (col >= a.width) return;
    const int64_t n = a.index.n;
    const uint2* sorted = s.sorted + m * n;
    const int64_t p0 = chunk * s.chunk;
    const int64_t p1 = p0 + s.chunk < n ? p0 + s.chunk : n;
    uint32_t cur = sorted[p0].x;
    if (cur == kNone) return;
    bool began_before = p0 > 0 && sorted[p0 - 1].x == cur;
    float* part = s.part + (m * s.chunks + chunk) * 2 * a.width;
    float acc[U * VEC];
#pragma unroll
    for (int e = 0; e < U * VEC; ++e) acc[e] = 0.f;
    auto put = [&](float* dst) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (col + u * step < a.width)
#pragma unroll
                for (int e = 0; e < VEC; ++e) dst[col + u * step + e] = acc[u * VEC + e];
    };
    for (int64_t p = p0; p < p1 && cur != kNone; p += B) {
        uint32_t key[B], tok[B];
        bool on[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const uint2 kt = p + j < p1 ? sorted[p + j] : make_uint2(kNone, 0u);
            key[j] = kt.x;
            on[j] = kt.x != kNone;
            tok[j] = on[j] ? kt.y : 0u;
        }
        float v[B][U * VEC];
        load_rows<T, VEC, U, B, CP>(a, m, tok, on, col, step, v);
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (p + j >= p1 || cur == kNone) break;
            if (key[j] != cur) {
                if (began_before) put(part);
                else write_row<TO, VEC, U>(a, m, cur, col, step, acc);
                began_before = false;
                cur = key[j];
#pragma unroll
                for (int e = 0; e < U * VEC; ++e) acc[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < U * VEC; ++e) acc[e] += v[j][e];
        }
    }
    if (cur == kNone) return;
    if (began_before) put(part);
    else if (p1 < n && sorted[p1].x == cur) put(part + a.width);
    else write_row<TO, VEC, U>(a, m, cur, col, step, acc);
}

// Adds the partial sums of the run that begins in chunk blockIdx.x and goes on in
// the next ones: warp w takes every 8th chunk, then the warps' sums are added in order.
template <typename TO>
__global__ void __launch_bounds__(kThreads) row_join_kernel(SumArgs s) {
    const RowSumArgs& a = s.a;
    const int m = blockIdx.z;
    const int64_t n = a.index.n, chunk = blockIdx.x;
    const uint2* sorted = s.sorted + m * n;
    const int64_t p0 = chunk * s.chunk, p1 = p0 + s.chunk;
    if (p1 >= n) return;
    const uint32_t key = sorted[p1 - 1].x;
    if (key == kNone || sorted[p1].x != key) return;
    if (p0 > 0 && sorted[p0 - 1].x == key) return;   // began in a chunk before
    // last chunk whose first token has this index
    int64_t lo = chunk + 1, hi = s.chunks - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (sorted[mid * s.chunk].x == key) lo = mid;
        else hi = mid - 1;
    }
    __shared__ float sums[kThreads / 32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = (int64_t)blockIdx.y * 32 + lane;
    const float* part = s.part + (int64_t)m * s.chunks * 2 * a.width;
    float acc = 0.f;
    if (col < a.width) {
        if (warp == 0) acc = part[(chunk * 2 + 1) * a.width + col];
        for (int64_t c = chunk + 1 + warp; c <= lo; c += kThreads / 32) acc += part[c * 2 * a.width + col];
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && col < a.width) {
        for (int w = 1; w < kThreads / 32; ++w) acc += sums[w][lane];
        write_row<TO, 1, 1>(a, m, key, col, 0, &acc);
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

template <typename T>
cudaError_t lookup(const LookupArgs& a, int type, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    const bool w = wide(a.table, a.table_stride, a.width, type) && wide(a.out, a.out_stride, a.width, type);
    const int l = log2_lanes(w ? cdiv(a.width, kVec) : a.width);
    const unsigned blocks = (unsigned)cdiv(a.index.n << l, kThreads);
    if (w) lookup_kernel<T, kVec><<<blocks, kThreads, 0, s>>>(a, l);
    else lookup_kernel<T, 1><<<blocks, kThreads, 0, s>>>(a, l);
    return cudaGetLastError();
}

template <typename T, typename TO, bool CP>
cudaError_t sums(const SumArgs& s, bool w, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T), kU = 8 / kVec, kB = CP ? 4 : 8;
    const int64_t groups = kThreads >> s.log2L;
    const dim3 grid((unsigned)cdiv(s.chunks, groups), (unsigned)cdiv(s.a.width, (int64_t)8 << s.log2L), s.a.index.d);
    if (w) row_sum_kernel<T, TO, kVec, kU, kB, CP><<<grid, kThreads, 0, st>>>(s);
    else row_sum_kernel<T, TO, 1, 8, kB, CP><<<grid, kThreads, 0, st>>>(s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || s.chunks < 2) return e;
    const dim3 join((unsigned)s.chunks, (unsigned)cdiv(s.a.width, 32), s.a.index.d);
    row_join_kernel<TO><<<join, kThreads, 0, st>>>(s);
    return cudaGetLastError();
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

// tokens a chunk: enough chunks to fill the GPU, at most 256 tokens each
int chunk_tokens(int64_t n) {
    int c = 8;
    while (c < 256 && n / c > 4096) c *= 2;
    return c;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, int type, cudaStream_t s) {
    if (a.index.n == 0) return cudaSuccess;
    if (type == MTTKRP_F32) return lookup<float>(a, type, s);
    if (type == MTTKRP_BF16) return lookup<__nv_bfloat16>(a, type, s);
    return lookup<__half>(a, type, s);
}

size_t row_sum_workspace_bytes(int64_t n, int d, int64_t width) {
    const int64_t chunks = cdiv(n, chunk_tokens(n));
    return 2 * align256(sizeof(uint2) * d * n) + sizeof(float) * d * chunks * 2 * width;
}

cudaError_t launch_row_sum(const RowSumArgs& a, cudaStream_t s) {
    const int64_t n = a.index.n;
    const int d = a.index.d;
    if (!a.accumulate) {
        const size_t e = elem_bytes(a.out_type);
        for (int m = 0; m < d; ++m) {
            cudaError_t err = cudaMemset2DAsync(a.out[m], a.out_stride * e, 0, a.width * e, a.index.rows[m], s);
            if (err != cudaSuccess) return err;
        }
    }
    if (n == 0) return cudaSuccess;
    SortArgs so;
    so.index = a.index;
    so.buf[0] = static_cast<uint2*>(a.ws);
    so.buf[1] = reinterpret_cast<uint2*>(static_cast<char*>(a.ws) + align256(sizeof(uint2) * d * n));
    // digits cover the indices and, above them, one value for tokens that take no part
    int64_t most = 0;
    for (int m = 0; m < d; ++m) most = a.index.rows[m] > most ? a.index.rows[m] : most;
    int bits = 1;
    while (((int64_t)1 << bits) <= most) ++bits;
    so.passes = (int)cdiv(bits, kMaxDigit);
    so.bits = (int)cdiv(bits, so.passes);
    so.first = (so.passes & 1) ? 1 : 0;
    const size_t smem = sizeof(uint32_t) * ((kSortWarps + 1) * ((size_t)1 << so.bits) + kSortWarps);
    static bool set = false;
    if (!set) {
        cudaError_t err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               sizeof(uint32_t) * ((kSortWarps + 1) * (1 << kMaxDigit) + kSortWarps));
        if (err != cudaSuccess) return err;
        set = true;
    }
    sort_kernel<<<kCluster * d, kSortThreads, smem, s>>>(so);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;

    SumArgs su;
    su.a = a;
    su.sorted = so.buf[1];
    su.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + 2 * align256(sizeof(uint2) * d * n));
    su.chunk = chunk_tokens(n);
    su.chunks = cdiv(n, su.chunk);
    su.log2L = log2_lanes(cdiv(a.width, 8));
    const bool cp = a.grad == nullptr;
    bool w = cp || wide(a.grad, a.grad_stride, a.width, a.type);
    for (int m = 0; m < d; ++m) {
        // results are written in vectors of as many elements as the rows are read in
        const size_t vec_bytes = 16 / elem_bytes(a.type) * elem_bytes(a.out_type);
        w = w && (reinterpret_cast<uintptr_t>(a.out[m]) % vec_bytes) == 0 &&
            (a.out_stride * elem_bytes(a.out_type)) % vec_bytes == 0;
        if (cp) w = w && wide(a.factor[m], a.width, a.width, a.type);
    }
    using bf16 = __nv_bfloat16;
    if (cp) {
        if (a.type == MTTKRP_F32) return sums<float, float, true>(su, w, s);
        if (a.type == MTTKRP_BF16) return sums<bf16, float, true>(su, w, s);
        return sums<__half, float, true>(su, w, s);
    }
    if (a.type == MTTKRP_F32) return sums<float, float, false>(su, w, s);
    if (a.type == MTTKRP_BF16)
        return a.out_type == MTTKRP_F32 ? sums<bf16, float, false>(su, w, s) : sums<bf16, bf16, false>(su, w, s);
    return a.out_type == MTTKRP_F32 ? sums<__half, float, false>(su, w, s) : sums<__half, __half, false>(su, w, s);
}

cudaError_t launch_entries(const EntriesArgs& a, int type, cudaStream_t s) {
    if (a.index.n == 0) return cudaSuccess;
    if (type == MTTKRP_F32) return entries<float>(a, type, s);
    if (type == MTTKRP_BF16) return entries<__nv_bfloat16>(a, type, s);
    return entries<__half>(a, type, s);
}

}  // namespace mk
