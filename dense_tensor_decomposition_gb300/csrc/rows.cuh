// Device helpers of the operators on rows: indices, scans.
#pragma once

#include <atomic>
#include <type_traits>

#include "launch.cuh"
#include "sort.h"
#include "types.cuh"

namespace mk {

__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr size_t elem_bytes(int type) { return type == MTTKRP_F32 ? 4 : 2; }

constexpr int kSms = 152;       // of a GB300; what a process is given may be fewer

// Dynamic shared memory that a CTA may ask for, of the 227 KB that it can have.
constexpr size_t kMaxSmem = 226 * 1024;

// lets a kernel have that much on the current device
template <auto kernel>
cudaError_t allow_smem() {
    static std::atomic<uint64_t> done{0};       // a bit a device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1) != 0)) return e;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kMaxSmem - attr.sharedSizeBytes));
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    return e;
}

__device__ __forceinline__ int64_t index_at(const IndexArgs& a, int64_t t, int m) {
    const int64_t at = t * a.stride + m;
    return a.bytes == 8 ? static_cast<const int64_t*>(a.idx)[at] : (int64_t) static_cast<const int32_t*>(a.idx)[at];
}

// the row that token t points to in column m, kNone where it takes no part; the loads
// of all columns (at most kCols) are issued together
template <typename I, int kCols>
__device__ __forceinline__ uint32_t sort_key_of(const IndexArgs& a, int64_t t, int m) {
    using U = std::make_unsigned_t<I>;
    const I* idx = static_cast<const I*>(a.idx) + t * a.stride;
    I v[kCols];
#pragma unroll
    for (int l = 0; l < kCols; ++l) v[l] = l < a.d ? idx[l] : 0;
    uint32_t key = 0;
    bool inside = true;
#pragma unroll
    for (int l = 0; l < kCols; ++l) {
        inside &= l >= a.d || (U)v[l] < (U)a.rows[l];       // negative: above every row
        key = l == m ? (uint32_t)v[l] : key;
    }
    return inside ? key : kNone;
}

template <typename I, int kCols>
struct KeyOf {
    static constexpr int kLook = kCols == 1 ? 8 : kCols <= 5 ? 4 : 2;       // tokens whose loads fit the registers
    __device__ __forceinline__ uint32_t operator()(const IndexArgs& a, int64_t t, int m) const {
        return sort_key_of<I, kCols>(a, t, m);
    }
};

// calls f with the KeyOf for these indices: loops over tokens go inside f, so that
// nothing stands between the loads of several tokens
template <typename F>
__device__ __forceinline__ void with_key(const IndexArgs& a, const F& f) {
    if (a.d == 1) a.bytes == 8 ? f(KeyOf<int64_t, 1>()) : f(KeyOf<int32_t, 1>());
    else if (a.d <= 3) a.bytes == 8 ? f(KeyOf<int64_t, 3>()) : f(KeyOf<int32_t, 3>());
    else if (a.d <= 5) a.bytes == 8 ? f(KeyOf<int64_t, 5>()) : f(KeyOf<int32_t, 5>());
    else a.bytes == 8 ? f(KeyOf<int64_t, MTTKRP_MAX_ORDER>()) : f(KeyOf<int32_t, MTTKRP_MAX_ORDER>());
}

__device__ __forceinline__ uint32_t sort_key(const IndexArgs& a, int64_t t, int m) {
    uint32_t key = kNone;
    with_key(a, [&](auto key_of) { key = key_of(a, t, m); });
    return key;
}

// Sum of x over the threads before this one of the first kWarps warps of a CTA, which
// sync() makes wait for one another, and over all (in `all`); sums: one word a warp.
// The threads wait twice.
template <int kWarps, typename Sync>
__device__ __forceinline__ uint32_t scan_warps(uint32_t x, uint32_t* sums, uint32_t& all, const Sync& sync) {
    static_assert(kWarps <= 32, "a lane for each warp");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t scan = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += up;
    }
    sync();
    if (lane == 31) sums[warp] = scan;
    sync();
    const uint32_t w = lane < kWarps ? sums[lane] : 0;
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

// row of a group's table for the sample at token t
__device__ __forceinline__ uint32_t table_row(const IndexArgs& a, const Tables::Group& g, int64_t t) {
    uint32_t row = 0;
    for (int k = 0; k < g.modes; ++k)
        row = row * (uint32_t)a.rows[g.mode[k]] + (uint32_t)index_at(a, t, g.mode[k]);
    return g.first + row;
}

}  // namespace mk
