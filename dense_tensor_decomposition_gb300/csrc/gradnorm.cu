// Norm over many tensors, and clipping by it:
//   norm = sqrt(sum over all tensors and elements of x^2),
//   y = x * min(1, max_norm / (norm + eps)).
//
// Bound by memory: 2 reads and 1 write of every element, less what of the first
// read is still in the L2 cache at the second.  The tensors are described in the
// kernel's arguments and cut into units of 8 KB; every block takes consecutive units,
// so each of the GPU's blocks has the same bytes to move whatever the tensors' sizes.
// One launch adds the squares and leaves a sum a block; in a second one every block adds
// the blocks' sums, in the same order, and multiplies its share, from the last unit back
// to the first (the last ones are the ones still cached: reads that will not be
// repeated and all writes are marked for the cache to drop first).  One cooperative
// launch with a barrier over the grid instead takes 12.3 us for 3 x 512 x 2000 fp32,
// the two, of which the second is set up while the first runs, 10.3 us; more blocks than
// are resident at once, for the SMs to take as they get free, lose the cache's order
// (192 MB of bf16: 112 us against 93).  More tensors than a table holds take both
// launches for each table.
//
// The squares of 16 elements are added in fp32, the sums of 16 in pairs of fp32 numbers
// (the second holds what the first rounds away): fp64 additions would take longer than
// the reads, at 2 a cycle and SM.
#include <atomic>

#include "launch.cuh"
#include "rows.h"
#include "squares.cuh"
#include "types.cuh"

namespace mk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;                          // 16-byte vectors a thread has in flight, a unit each
constexpr int kUnitVecs = kThreads;                 // 8 KB
constexpr int kLog2UnitBytes = 13;
static_assert(kUnitVecs * 16 == 1 << kLog2UnitBytes);
constexpr int kMaxBlocks = 2048;                    // most sums a table
constexpr int64_t kCached = 64 << 20;               // bytes of the first read to find in L2 at the second
constexpr int kSmallTable = 32, kMiddleTable = 400, kLargeTable = 1024;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 29 bytes a tensor: the large table is just below the 32764 bytes that a
// kernel's arguments can hold, the others spare shorter lists its copy.  (By the middle
// table and by the large one: 100 tensors 10.5 and 11.6 us, 400 tensors of 64 elements
// 19.0 and 21.0, of 250000 65.6 and 69.9; by the small one and by the middle one, 32
// tensors 8.1 and 8.2 us.)
template <int N>
struct Table {
    const void* in[N];
    void* out[N];
    int64_t numel[N];
    uint32_t first[N];      // number of the tensor's first unit
    uint8_t type[N];
    int n;
    uint32_t units;
};

// Vectors of a tensor start at multiples of 16 bytes, the first one at or before
// its first element; elements before the first or behind the last are not touched.
template <typename T>
struct Vecs {
    static constexpr int kVec = 16 / sizeof(T);
    using P = Pack<T, kVec>;
    const T* x;
    int64_t n;
    int shift;              // elements of the first vector that lie before x
    __device__ Vecs(const void* p, int64_t numel)
        : x(static_cast<const T*>(p)), n(numel), shift((int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T)) {}
    __device__ bool whole(int64_t i) const { return i * kVec >= shift && (i + 1) * kVec - shift <= n; }
    __device__ bool holds(int64_t e) const { return e >= 0 && e < n; }
    __device__ const uint4* at(int64_t i) const { return reinterpret_cast<const uint4*>(x - shift) + i; }
    // zeros for elements that are not the tensor's
    __device__ uint4 load(int64_t i) const {
        if (whole(i)) return *at(i);
        P v;
#pragma unroll
        for (int e = 0; e < kVec; ++e) v.v[e] = holds(i * kVec - shift + e) ? x[i * kVec - shift + e] : from_f32<T>(0.f);
        return as_pack<uint4>(v);
    }
    // vectors i, i + kUnitVecs, ... of `units` <= kUnroll units; keep: for the cache to keep
    __device__ void load_units(int64_t i, int units, bool keep, uint4* v) const {
        if (units == kUnroll && whole(i - threadIdx.x) && whole(i - threadIdx.x + (int64_t)kUnroll * kUnitVecs - 1)) {
            if (keep) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) v[u] = *at(i + u * kUnitVecs);
            } else {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) v[u] = __ldcs(at(i + u * kUnitVecs));
            }
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) v[u] = u < units ? load(i + u * kUnitVecs) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
};

template <typename T>
__device__ __forceinline__ void add_squares(const void* p, int64_t numel, int64_t unit, int units, bool keep, Sum& sum) {
    constexpr int kVec = Vecs<T>::kVec;
    const Vecs<T> x(p, numel);
    uint4 v[kUnroll];
    x.load_units(unit * kUnitVecs + threadIdx.x, units, keep, v);
#pragma unroll
    for (int u = 0; u < kUnroll; u += 16 / kVec) {
        float f[16];
#pragma unroll
        for (int w = 0; w < 16 / kVec; ++w) {
            const Pack<T, kVec> p = as_pack<Pack<T, kVec>>(v[u + w]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[w * kVec + e] = to_f32(p.v[e]);
        }
        sum.squares16(f);
    }
}

template <typename T>
__device__ __forceinline__ void scale(const void* p, void* q, int64_t numel, int64_t unit, int units, float coef) {
    constexpr int kVec = Vecs<T>::kVec;
    const Vecs<T> x(p, numel);
    T* y = static_cast<T*>(q);
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    const int64_t i = unit * kUnitVecs + threadIdx.x;
    uint4 v[kUnroll];
    x.load_units(i, units, false, v);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= units) break;
        const int64_t at = i + u * kUnitVecs, e0 = at * kVec - x.shift;
        auto w = as_pack<Pack<T, kVec>>(v[u]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) w.v[e] = from_f32<T>(coef * to_f32(w.v[e]));
        if (same && x.whole(at)) {
            __stcs(reinterpret_cast<uint4*>(y + e0), as_pack<uint4>(w));
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (x.holds(e0 + e)) y[e0 + e] = w.v[e];
        }
    }
}

// the tensor that a unit is of: the last one whose first unit is not above it
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& a, uint32_t unit) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= unit) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// this block's share of the units
template <int N>
__device__ __forceinline__ void share(const Table<N>& a, uint32_t& t0, uint32_t& t1) {
    t0 = (uint32_t)((uint64_t)a.units * blockIdx.x / gridDim.x);
    t1 = (uint32_t)((uint64_t)a.units * (blockIdx.x + 1) / gridDim.x);
}

template <int N>
__device__ __forceinline__ double share_squares(const Table<N>& a) {
    uint32_t t0, t1;
    share(a, t0, t1);
    // the last ones are read again first
    const uint32_t kept = (uint32_t)(kCached / (kUnitVecs * 16)) / gridDim.x;
    const uint32_t keep_from = t1 - t0 > kept ? t1 - kept : t0;
    Sum sum;
    int k = t0 < t1 ? tensor_of(a, t0) : 0;
    for (uint32_t t = t0; t < t1;) {
        while (k + 1 < a.n && a.first[k + 1] <= t) ++k;
        const uint32_t end = k + 1 < a.n && a.first[k + 1] < t1 ? a.first[k + 1] : t1;
        const int units = end - t < kUnroll ? (int)(end - t) : kUnroll;
        const uint32_t at = t - a.first[k];
        const bool keep = t >= keep_from;
        if (a.type[k] == MTTKRP_F32) add_squares<float>(a.in[k], a.numel[k], at, units, keep, sum);
        else if (a.type[k] == MTTKRP_BF16) add_squares<__nv_bfloat16>(a.in[k], a.numel[k], at, units, keep, sum);
        else add_squares<__half>(a.in[k], a.numel[k], at, units, keep, sum);
        t += units;
    }
    return block_sum<kWarps>(sum);
}

template <int N>
__device__ __forceinline__ void share_scale(const Table<N>& a, float coef) {
    uint32_t t0, t1;
    share(a, t0, t1);
    int k = t0 < t1 ? tensor_of(a, t1 - 1) : 0;
    for (uint32_t t = t1; t > t0;) {
        while (a.first[k] >= t) --k;
        const uint32_t begin = a.first[k] > t0 ? a.first[k] : t0;
        const int units = t - begin < kUnroll ? (int)(t - begin) : kUnroll;
        t -= units;
        if (coef == 1.f && a.in[k] == a.out[k]) continue;       // nothing changes
        const uint32_t at = t - a.first[k];
        if (a.type[k] == MTTKRP_F32) scale<float>(a.in[k], a.out[k], a.numel[k], at, units, coef);
        else if (a.type[k] == MTTKRP_BF16) scale<__nv_bfloat16>(a.in[k], a.out[k], a.numel[k], at, units, coef);
        else scale<__half>(a.in[k], a.out[k], a.numel[k], at, units, coef);
    }
}

// The norm from the blocks' sums, by one warp, and the coefficient (which follows the
// formula for infinite and NaN norms too: 0 and NaN).
struct Norm {
    float norm, coef;
};

__device__ __forceinline__ Norm norm_of(const double* part, int n, float max_norm, float eps) {
    __shared__ Norm found;
    if (threadIdx.x < 32) {
        double sum = 0.0;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += 32) sum += part[i];
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (threadIdx.x == 0) {
            Norm r;
            if (sum >= 0x1p-100 && sum <= 0x1p100) {        // fp32 will do
                r.norm = sqrtf((float)sum);
                const float c = max_norm / (r.norm + eps);
                r.coef = c >= 1.f ? 1.f : c;
            } else {
                const double root = sqrt(sum), c = (double)max_norm / (root + (double)eps);
                r.norm = (float)root;
                r.coef = c >= 1.0 ? 1.f : (float)c;
            }
            found = r;
        }
    }
    __syncthreads();
    return found;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 2) squares_kernel(const __grid_constant__ Table<N> a, double* part) {
    after_previous();
    const double sum = share_squares(a);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 2) scale_kernel(const __grid_constant__ Table<N> a, const double* part,
                                                            int parts, float max_norm, float eps, float* norm) {
    after_previous();
    const Norm r = norm_of(part, parts, max_norm, eps);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r.norm;
    share_scale(a, r.coef);
}

// the norm alone
__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int parts, float* norm) {
    after_previous();
    const Norm r = norm_of(part, parts, 0.f, 0.f);
    if (threadIdx.x == 0) *norm = r.norm;
}

// blocks of a launch that are resident at once on the current device
template <int N>
cudaError_t resident_blocks(int& blocks) {
    static std::atomic<int> cached[64];     // by device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && cached[dev] > 0) {
        blocks = cached[dev];
        return cudaSuccess;
    }
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, scale_kernel<N>, kThreads, 0);
    if (e != cudaSuccess) return e;
    blocks = sms * per_sm < kMaxBlocks ? sms * per_sm : kMaxBlocks;
    if (dev < 64) cached[dev] = blocks;
    return cudaSuccess;
}

// One table of at most N tensors, starting at tensor k; returns how many it took
// (tensors without elements are left out of the table).
template <int N>
int fill(Table<N>& t, int n, int k, const void* const* tensors, const int64_t* numels, const int* types,
         void* const* outs) {
    int used = 0;
    int64_t units = 0;
    t.n = 0;
    for (; k + used < n && t.n < N; ++used) {
        const int i = k + used;
        if (numels[i] == 0) continue;
        t.in[t.n] = tensors[i];
        t.out[t.n] = outs ? outs[i] : nullptr;
        t.numel[t.n] = numels[i];
        t.type[t.n] = (uint8_t)types[i];
        t.first[t.n] = (uint32_t)units;
        // elements from the first vector's start, in units (by shifts: about 200 tensors a call)
        const int shift = types[i] == MTTKRP_F32 ? 2 : 1;
        const int64_t to = numels[i] + (int64_t)((reinterpret_cast<uintptr_t>(tensors[i]) & 15) >> shift);
        const int64_t unit = kUnitVecs * 16 >> shift;
        units += (to + unit - 1) >> (kLog2UnitBytes - shift);
        ++t.n;
    }
    t.units = (uint32_t)units;
    return used;
}

template <int N>
cudaError_t norm_and_clip(int n, const void* const* tensors, const int64_t* numels, const int* types,
                          void* const* outs, float max_norm, float eps, float* norm, void* ws, cudaStream_t s) {
    double* part = static_cast<double*>(ws);
    int most = 0;
    cudaError_t e = resident_blocks<N>(most);
    auto blocks = [&](const Table<N>& t) { return t.units < (uint32_t)most ? (int)t.units : most; };
    Table<N> t;
    int parts = 0, tables = 0;
    for (int k = 0; k < n && e == cudaSuccess; ++tables) {
        k += fill(t, n, k, tensors, numels, types, outs);
        if (t.units == 0) continue;
        e = launch_early(squares_kernel<N>, blocks(t), kThreads, 0, s, t, part + parts);
        parts += blocks(t);
    }
    if (e != cudaSuccess) return e;
    if (!outs || parts == 0) return launch_early(norm_kernel, 1, kThreads, 0, s, part, parts, norm);
    for (int k = 0; k < n && e == cudaSuccess;) {
        k += tables == 1 ? n : fill(t, n, k, tensors, numels, types, outs);
        if (t.units > 0)
            e = launch_early(scale_kernel<N>, blocks(t), kThreads, 0, s, t, part, parts, max_norm, eps, norm);
    }
    return e;
}

}  // namespace

// at most kMaxBlocks sums a table
size_t grad_norm_workspace_bytes(int n) {
    const int64_t tables = n <= kSmallTable ? 1 : cdiv(n, kLargeTable);
    return sizeof(double) * kMaxBlocks * tables;
}

cudaError_t launch_grad_norm(int n, const void* const* tensors, const int64_t* numels, const int* types,
                             void* const* outs, float max_norm, float eps, float* norm, void* ws,
                             cudaStream_t s) {
    if (n <= kSmallTable)
        return norm_and_clip<kSmallTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
    if (n <= kMiddleTable)
        return norm_and_clip<kMiddleTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
    return norm_and_clip<kLargeTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
}

}  // namespace mk
