// Norm over many tensors, and clipping by it:
//   norm = sqrt(sum over all tensors and elements of x^2),
//   y = x * min(1, max_norm / (norm + eps)).
//
// Bound by memory: 2 reads and 1 write of every element, less what of the first
// read is still in the L2 cache at the second.  The tensors are described in the
// kernel's arguments and cut into 16 KB tiles; every block takes consecutive
// tiles, so each of the GPU's blocks has the same bytes to move whatever the
// tensors' sizes.  One cooperative launch does it all: squares, a barrier over the
// grid, every block adds the blocks' sums in the same order, then the products,
// from the last tile back to the first (the last ones are the ones still cached).
// More tensors than a table holds take one launch a table and step.
#include <cooperative_groups.h>

#include "rows.h"
#include "types.cuh"

namespace cg = cooperative_groups;

namespace mk {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                          // 16-byte vectors a thread has in flight
constexpr int kTileVecs = kThreads * kUnroll;       // 16 KB
constexpr int kMaxBlocks = 2048;
constexpr int kSmallTable = 32, kLargeTable = 1024;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 29 bytes a tensor: the large table is just below the 32764 bytes that a
// kernel's arguments can hold, the small one spares short lists its copy.
template <int N>
struct Table {
    const void* in[N];
    void* out[N];
    int64_t numel[N];
    uint32_t first[N];      // number of the tensor's first tile
    uint8_t type[N];
    int n;
    uint32_t tiles;
};

// Vectors of a tensor start at multiples of 16 bytes, the first one at or before
// its first element; elements before the first or behind the last are not touched.
template <typename T>
struct Vecs {
    static constexpr int kVec = 16 / sizeof(T);
    const T* x;
    int64_t n;
    int shift;              // elements of the first vector that lie before x
    __device__ Vecs(const void* p, int64_t numel)
        : x(static_cast<const T*>(p)), n(numel), shift((int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T)) {}
    __device__ bool whole(int64_t i) const { return i * kVec >= shift && (i + 1) * kVec - shift <= n; }
    __device__ bool holds(int64_t e) const { return e >= 0 && e < n; }
    __device__ Pack<T, kVec> load(int64_t i) const {
        const int64_t e0 = i * kVec - shift;
        if (whole(i)) return *reinterpret_cast<const Pack<T, kVec>*>(x + e0);
        Pack<T, kVec> v;
#pragma unroll
        for (int e = 0; e < kVec; ++e) v.v[e] = holds(e0 + e) ? x[e0 + e] : from_f32<T>(0.f);
        return v;
    }
};

__device__ __forceinline__ double block_sum(double x) {
    __shared__ double sums[kThreads / 32];
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) x += sums[w];
    __syncthreads();
    return x;
}

// Sum of 16 squares in fp32; where it leaves the fp32 range, or is so small that
// fp32 drops bits of it, the same sum in fp64.
__device__ __forceinline__ double squares16(const float* v) {
    float s = 0.f, most = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        s = fmaf(v[e], v[e], s);
        most = fmaxf(most, fabsf(v[e]));
    }
    if ((s >= 0x1p-100f && s <= 0x1p127f) || (s == 0.f && most == 0.f)) return (double)s;
    double d = 0.0;
#pragma unroll
    for (int e = 0; e < 16; ++e) d = fma((double)v[e], (double)v[e], d);
    return d;
}

template <typename T>
__device__ __forceinline__ double tile_squares(const void* p, int64_t numel, uint32_t tile) {
    constexpr int kVec = Vecs<T>::kVec, kVecs16 = 16 / kVec;
    const Vecs<T> x(p, numel);
    const int64_t i0 = (int64_t)tile * kTileVecs + threadIdx.x;
    Pack<T, kVec> v[kUnroll];
    if (x.whole((int64_t)tile * kTileVecs) && x.whole((int64_t)(tile + 1) * kTileVecs - 1)) {
        const Pack<T, kVec>* src = reinterpret_cast<const Pack<T, kVec>*>(x.x - x.shift) + i0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = src[u * kThreads];
    } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = x.load(i0 + u * kThreads);
    }
    double sum = 0.0;
#pragma unroll
    for (int u = 0; u < kUnroll; u += kVecs16) {
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = to_f32(v[u + e / kVec].v[e % kVec]);
        sum += squares16(f);
    }
    return sum;
}

template <typename T>
__device__ __forceinline__ void tile_scale(const void* p, void* q, int64_t numel, uint32_t tile, float coef) {
    constexpr int kVec = Vecs<T>::kVec;
    const Vecs<T> x(p, numel);
    T* y = static_cast<T*>(q);
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    const int64_t i0 = (int64_t)tile * kTileVecs + threadIdx.x;
    Pack<T, kVec> v[kUnroll];
    if (same && x.whole((int64_t)tile * kTileVecs) && x.whole((int64_t)(tile + 1) * kTileVecs - 1)) {
        const Pack<T, kVec>* src = reinterpret_cast<const Pack<T, kVec>*>(x.x - x.shift) + i0;
        Pack<T, kVec>* dst = reinterpret_cast<Pack<T, kVec>*>(y - x.shift) + i0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = src[u * kThreads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[u].v[e] = from_f32<T>(coef * to_f32(v[u].v[e]));
            dst[u * kThreads] = v[u];
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = x.load(i0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t e0 = (i0 + u * kThreads) * kVec - x.shift;
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[u].v[e] = from_f32<T>(coef * to_f32(v[u].v[e]));
        if (same && x.whole(i0 + u * kThreads)) {
            *reinterpret_cast<Pack<T, kVec>*>(y + e0) = v[u];
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (x.holds(e0 + e)) y[e0 + e] = v[u].v[e];
        }
    }
}

// the tensor that a tile is of: the last one whose first tile is not above it
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& a, uint32_t tile) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// this block's share of the tiles
template <int N>
__device__ __forceinline__ void share(const Table<N>& a, uint32_t& t0, uint32_t& t1) {
    t0 = (uint32_t)((uint64_t)a.tiles * blockIdx.x / gridDim.x);
    t1 = (uint32_t)((uint64_t)a.tiles * (blockIdx.x + 1) / gridDim.x);
}

template <int N>
__device__ __forceinline__ double share_squares(const Table<N>& a) {
    uint32_t t0, t1;
    share(a, t0, t1);
    double sum = 0.0;
    int k = t0 < t1 ? tensor_of(a, t0) : 0;
    for (uint32_t t = t0; t < t1; ++t) {
        while (k + 1 < a.n && a.first[k + 1] <= t) ++k;
        const uint32_t at = t - a.first[k];
        if (a.type[k] == MTTKRP_F32) sum += tile_squares<float>(a.in[k], a.numel[k], at);
        else if (a.type[k] == MTTKRP_BF16) sum += tile_squares<__nv_bfloat16>(a.in[k], a.numel[k], at);
        else sum += tile_squares<__half>(a.in[k], a.numel[k], at);
    }
    return block_sum(sum);
}

template <int N>
__device__ __forceinline__ void share_scale(const Table<N>& a, float coef) {
    uint32_t t0, t1;
    share(a, t0, t1);
    int k = t0 < t1 ? tensor_of(a, t1 - 1) : 0;
    for (uint32_t t = t1; t-- > t0;) {
        while (a.first[k] > t) --k;
        if (coef == 1.f && a.in[k] == a.out[k]) continue;       // nothing changes
        const uint32_t at = t - a.first[k];
        if (a.type[k] == MTTKRP_F32) tile_scale<float>(a.in[k], a.out[k], a.numel[k], at, coef);
        else if (a.type[k] == MTTKRP_BF16) tile_scale<__nv_bfloat16>(a.in[k], a.out[k], a.numel[k], at, coef);
        else tile_scale<__half>(a.in[k], a.out[k], a.numel[k], at, coef);
    }
}

// The norm from the blocks' sums, and the coefficient (which follows the formula
// for infinite and NaN norms too: 0 and NaN).
__device__ __forceinline__ float norm_of(const double* part, int n, float max_norm, float eps, float& norm) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) sum += __ldcg(part + i);
    const double r = sqrt(block_sum(sum));
    norm = (float)r;
    const double c = (double)max_norm / (r + (double)eps);
    return c >= 1.0 ? 1.f : (float)c;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) clip_kernel(const __grid_constant__ Table<N> a, double* part,
                                                           float max_norm, float eps, float* norm) {
    const double sum = share_squares(a);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
    cg::this_grid().sync();
    float r;
    const float coef = norm_of(part, gridDim.x, max_norm, eps, r);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
    share_scale(a, coef);
}

// the same steps as launches of their own
template <int N>
__global__ void __launch_bounds__(kThreads, 4) squares_kernel(const __grid_constant__ Table<N> a, double* part) {
    const double sum = share_squares(a);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int n, float max_norm, float eps,
                                                        float* norm, float* coef) {
    float r;
    const float c = norm_of(part, n, max_norm, eps, r);
    if (threadIdx.x == 0) {
        *norm = r;
        *coef = c;
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) scale_kernel(const __grid_constant__ Table<N> a, const float* coef) {
    share_scale(a, *coef);
}

// blocks of clip_kernel<N> that are resident at once on the current device
template <int N>
cudaError_t resident_blocks(int& blocks) {
    static int cached[64];      // by device; writing the same value twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && cached[dev] > 0) {
        blocks = cached[dev];
        return cudaSuccess;
    }
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, clip_kernel<N>, kThreads, 0);
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
    int64_t tiles = 0;
    t.n = 0;
    for (; k + used < n && t.n < N; ++used) {
        const int i = k + used;
        if (numels[i] == 0) continue;
        t.in[t.n] = tensors[i];
        t.out[t.n] = outs ? outs[i] : nullptr;
        t.numel[t.n] = numels[i];
        t.type[t.n] = (uint8_t)types[i];
        t.first[t.n] = (uint32_t)tiles;
        const int e = types[i] == MTTKRP_F32 ? 4 : 2;
        tiles += cdiv(numels[i] + (int64_t)(reinterpret_cast<uintptr_t>(tensors[i]) & 15) / e, kTileVecs * 16 / e);
        ++t.n;
    }
    t.tiles = (uint32_t)tiles;
    return used;
}

template <int N>
cudaError_t norm_and_clip(int n, const void* const* tensors, const int64_t* numels, const int* types,
                          void* const* outs, float max_norm, float eps, float* norm, void* ws, cudaStream_t s) {
    float* coef = static_cast<float*>(ws);
    double* part = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
    int most = 0;
    cudaError_t e = resident_blocks<N>(most);
    if (e != cudaSuccess) return e;
    auto blocks = [&](const Table<N>& t) { return t.tiles < (uint32_t)most ? (int)t.tiles : most; };
    Table<N> t;
    int k = fill(t, n, 0, tensors, numels, types, outs);
    if (outs && k == n && t.tiles > 0) {
        void* args[] = {&t, &part, &max_norm, &eps, &norm};
        return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(clip_kernel<N>), dim3(blocks(t)),
                                           dim3(kThreads), args, 0, s);
    }
    int parts = 0;
    for (;;) {
        if (t.tiles > 0) squares_kernel<N><<<blocks(t), kThreads, 0, s>>>(t, part + parts);
        parts += blocks(t);
        if (k == n) break;
        k += fill(t, n, k, tensors, numels, types, outs);
    }
    norm_kernel<<<1, kThreads, 0, s>>>(part, parts, max_norm, eps, norm, coef);
    for (k = 0; outs && k < n;) {
        k += fill(t, n, k, tensors, numels, types, outs);
        if (t.tiles > 0) scale_kernel<N><<<blocks(t), kThreads, 0, s>>>(t, coef);
    }
    return cudaGetLastError();
}

}  // namespace

// the coefficient, then at most kMaxBlocks partial sums a table
size_t grad_norm_workspace_bytes(int n) {
    const int64_t tables = n <= kSmallTable ? 1 : cdiv(n, kLargeTable);
    return 256 + sizeof(double) * kMaxBlocks * tables;
}

cudaError_t launch_grad_norm(int n, const void* const* tensors, const int64_t* numels, const int* types,
                             void* const* outs, float max_norm, float eps, float* norm, void* ws,
                             cudaStream_t s) {
    if (n <= kSmallTable)
        return norm_and_clip<kSmallTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
    return norm_and_clip<kLargeTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
}

}  // namespace mk
