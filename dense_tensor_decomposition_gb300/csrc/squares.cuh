// Sums of squares: 16 in fp32, these sums as pairs of fp32 numbers, and what leaves fp32's
// range in fp64.
#pragma once

#include <cuda_runtime.h>

namespace mk {

// a sum as hi + lo, and in fp64 what does not fit fp32's range
struct Sum {
    float hi = 0.f, lo = 0.f;
    double wide = 0.0;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;     // s + rounding error = hi + x, exactly
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    // 16 squares; sums up to 2^90 can be added 2^36 times
    __device__ __forceinline__ void squares16(const float* v) {
        float s = 0.f, most = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            s = fmaf(v[e], v[e], s);
            most = fmaxf(most, fabsf(v[e]));
        }
        if ((s >= 0x1p-100f && s <= 0x1p90f) || (s == 0.f && most == 0.f)) {
            add(s);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) wide = fma((double)v[e], (double)v[e], wide);
        }
    }
};

// over the block; the result in thread 0
template <int kWarps>
__device__ __forceinline__ Sum block_total(Sum s) {
    __shared__ float hi[kWarps], lo[kWarps];
    __shared__ double wide[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool any = __syncthreads_or(s.wide != 0.0) != 0;      // NaN too
    for (int o = 16; o > 0; o >>= 1) {
        const float l = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
        s.add(__shfl_xor_sync(0xFFFFFFFFu, s.hi, o));
        s.lo += l;
        if (any) s.wide += __shfl_xor_sync(0xFFFFFFFFu, s.wide, o);
    }
    if (lane == 0) {
        hi[warp] = s.hi;
        lo[warp] = s.lo;
        wide[warp] = s.wide;
    }
    __syncthreads();
    Sum t;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w) {
            t.add(hi[w]);
            t.lo += lo[w];
            if (any) t.wide += wide[w];
        }
    }
    return t;
}

template <int kWarps>
__device__ __forceinline__ double block_sum(Sum s) {
    const Sum t = block_total<kWarps>(s);
    return threadIdx.x == 0 ? (double)t.hi + (double)t.lo + t.wide : 0.0;
}

}  // namespace mk
