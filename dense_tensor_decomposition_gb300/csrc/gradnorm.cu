// Norm over many tensors, and clipping by it:
//   norm = sqrt(sum over all tensors and elements of x^2),
//   y = x * min(1, max_norm / (norm + eps)).
//
// One kernel adds the squares (fp32 over a few elements, then fp64) and leaves
// one partial sum a block; one block adds those in order and writes the norm and
// the coefficient; one kernel multiplies.  The tensors are described in the
// kernels' arguments, a table of them a launch.
#include "rows.h"
#include "types.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 152 * 8;
constexpr int kGroup = 16;          // elements whose squares are added in fp32
constexpr int kTile = kThreads * 4 * kGroup;
constexpr int kSmallTable = 32, kLargeTable = 1024;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A tile is kTile consecutive elements of one tensor.  29 bytes a tensor: the
// large table is just below the 32764 bytes that a kernel's arguments can hold.
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

__device__ __forceinline__ double block_sum(double x) {
    __shared__ double sums[kThreads / 32];
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) x += sums[w];
    return x;
}

template <typename T>
__device__ __forceinline__ double tile_squares(const T* __restrict__ x, int n) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads * kGroup) {
        float v[kGroup];
#pragma unroll
        for (int e = 0; e < kGroup; ++e) v[e] = i + e * kThreads < n ? to_f32(x[i + e * kThreads]) : 0.f;
        float s = 0.f, any = 0.f;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            s = fmaf(v[e], v[e], s);
            any = fmaxf(any, fabsf(v[e]));
        }
        // squares that leave the fp32 range, or lose bits at its lower end: in fp64
        if (s >= 0x1p-100f && s <= 0x1p127f) {
            sum += (double)s;
        } else if (!(s == 0.f && any == 0.f)) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) sum = fma((double)v[e], (double)v[e], sum);
        }
    }
    return sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<N> a, double* part) {
    double sum = 0.0;
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int k = tensor_of(a, tile);
        const int64_t at = (int64_t)(tile - a.first[k]) * kTile;
        const int n = (int)(a.numel[k] - at < kTile ? a.numel[k] - at : kTile);
        if (a.type[k] == MTTKRP_F32) sum += tile_squares(static_cast<const float*>(a.in[k]) + at, n);
        else if (a.type[k] == MTTKRP_BF16) sum += tile_squares(static_cast<const __nv_bfloat16*>(a.in[k]) + at, n);
        else sum += tile_squares(static_cast<const __half*>(a.in[k]) + at, n);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// coef follows the formula for infinite and NaN norms too (0 and NaN)
__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int n, float max_norm, float eps,
                                                        float* norm, float* coef) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const double r = sqrt(sum);
        *norm = (float)r;
        const double c = (double)max_norm / (r + (double)eps);
        *coef = c >= 1.0 ? 1.f : (float)c;
    }
}

template <typename T>
__device__ __forceinline__ void tile_scale(const T* x, T* y, int n, float coef) {
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kThreads) y[i] = from_f32<T>(coef * to_f32(x[i]));
}

template <int N>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<N> a, const float* coef_at) {
    const float coef = *coef_at;
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int k = tensor_of(a, tile);
        if (coef == 1.f && a.in[k] == a.out[k]) continue;    // nothing changes
        const int64_t at = (int64_t)(tile - a.first[k]) * kTile;
        const int n = (int)(a.numel[k] - at < kTile ? a.numel[k] - at : kTile);
        if (a.type[k] == MTTKRP_F32)
            tile_scale(static_cast<const float*>(a.in[k]) + at, static_cast<float*>(a.out[k]) + at, n, coef);
        else if (a.type[k] == MTTKRP_BF16)
            tile_scale(static_cast<const __nv_bfloat16*>(a.in[k]) + at, static_cast<__nv_bfloat16*>(a.out[k]) + at, n,
                       coef);
        else
            tile_scale(static_cast<const __half*>(a.in[k]) + at, static_cast<__half*>(a.out[k]) + at, n, coef);
    }
}

int blocks_of(uint32_t tiles) { return tiles < kBlocks ? (int)tiles : kBlocks; }

// One group of at most N tensors, starting at tensor k; returns how many it took
// (tensors without elements are left out of the table).
template <int N>
int fill(Table<N>& t, int n, int k, const void* const* tensors, const int64_t* numels, const int* types,
         void* const* outs) {
    int used = 0;
    t.n = 0;
    int64_t tiles = 0;
    for (; k + used < n && t.n < N; ++used) {
        const int i = k + used;
        if (numels[i] == 0) continue;
        const int64_t more = cdiv(numels[i], kTile);
        t.in[t.n] = tensors[i];
        t.out[t.n] = outs ? outs[i] : nullptr;
        t.numel[t.n] = numels[i];
        t.type[t.n] = (uint8_t)types[i];
        t.first[t.n] = (uint32_t)tiles;
        tiles += more;
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
    Table<N> t;
    int parts = 0;
    for (int k = 0; k < n;) {
        k += fill(t, n, k, tensors, numels, types, outs);
        if (t.tiles == 0) continue;
        squares_kernel<N><<<blocks_of(t.tiles), kThreads, 0, s>>>(t, part + parts);
        parts += blocks_of(t.tiles);
    }
    norm_kernel<<<1, kThreads, 0, s>>>(part, parts, max_norm, eps, norm, coef);
    if (outs) {
        for (int k = 0; k < n;) {
            k += fill(t, n, k, tensors, numels, types, outs);
            if (t.tiles != 0) scale_kernel<N><<<blocks_of(t.tiles), kThreads, 0, s>>>(t, coef);
        }
    }
    return cudaGetLastError();
}

}  // namespace

// the coefficient, then at most kBlocks partial sums a launch
size_t grad_norm_workspace_bytes(int n) {
    const int64_t groups = n <= kSmallTable ? 1 : cdiv(n, kLargeTable);
    return 256 + sizeof(double) * kBlocks * groups;
}

cudaError_t launch_grad_norm(int n, const void* const* tensors, const int64_t* numels, const int* types,
                             void* const* outs, float max_norm, float eps, float* norm, void* ws,
                             cudaStream_t s) {
    if (n <= kSmallTable)
        return norm_and_clip<kSmallTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
    return norm_and_clip<kLargeTable>(n, tensors, numels, types, outs, max_norm, eps, norm, ws, s);
}

}  // namespace mk
