// What the kernels of the orthogonalisation share: lists of matrices, their elements, images
// (see newton.cu), U and its norm, and results.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "mttkrp.h"
#include "newton_plan.h"
#include "ptx.cuh"
#include "squares.cuh"
#include "types.cuh"

namespace mk {

constexpr uint32_t kTileBytes = 8192;
constexpr float kScale = 4096.f, kUnscale = 1.f / 4096.f;   // of the images

// Rows of a matrix in its own memory.
struct Store {
    void* data;
    int64_t row, batch;         // strides
    uint8_t type, whole;        // whole: eight elements from a multiple of eight on are aligned to 16 bytes
};

// Eight consecutive elements of a row as they lie in memory: 32 bytes, or 16 in x.
struct Raw8 {
    uint4 x, y;
};
// Those of row r from column c on; zeros from `cols` on.  (One piece of code for all types, which differ
// in how much of it they use: a copy a type is more instructions than the cache holds for as long as a
// kernel of a few microseconds runs.)  fast: all eight are there and aligned, or nothing is to be read (in).
__device__ __forceinline__ Raw8 raw_fast(const Store& s, bool in, int64_t b, int r, int c) {
    const bool wide = s.type == MTTKRP_F32;
    const uint8_t* p = static_cast<const uint8_t*>(s.data) + ((b * s.batch + r * s.row + c) << (wide ? 2 : 1));
    Raw8 w;
    w.x = w.y = make_uint4(0u, 0u, 0u, 0u);
    if (in) w.x = *reinterpret_cast<const uint4*>(p);
    if (in && wide) w.y = *reinterpret_cast<const uint4*>(p + 16);
    return w;
}
__device__ __forceinline__ Raw8 raw_any(const Store& s, bool in, int64_t b, int r, int c, int cols) {
    if (s.whole && c + 8 <= cols) return raw_fast(s, in, b, r, c);
    const int valid = in ? cols - c : 0;
    const int64_t at = b * s.batch + r * s.row + c;
    uint32_t w[8];
    if (s.type == MTTKRP_F32) {
        const uint32_t* p = static_cast<const uint32_t*>(s.data) + at;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < valid ? p[e] : 0u;
        return Raw8{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
    }
    const uint16_t* p = static_cast<const uint16_t*>(s.data) + at;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = e < valid ? (uint32_t)p[e] : 0u;
    return Raw8{make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16),
                make_uint4(0u, 0u, 0u, 0u)};
}
__device__ __forceinline__ void values(uint8_t type, const Raw8& w, float* v) {
    const uint32_t x[4] = {w.x.x, w.x.y, w.x.z, w.x.w}, y[4] = {w.y.x, w.y.y, w.y.z, w.y.w};
    if (type == MTTKRP_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(x[e]);
            v[4 + e] = __uint_as_float(y[e]);
        }
    } else if (type == MTTKRP_BF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(x[e] << 16);
            v[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}
__device__ __forceinline__ uint32_t pair16(bool bf16, float a, float b) {
    const __nv_bfloat162 f = __floats2bfloat162_rn(a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return bf16 ? *reinterpret_cast<const uint32_t*>(&f) : *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void put8(const Store& s, int64_t b, int r, int c, int cols, const float* v) {
    const int64_t at = b * s.batch + r * s.row + c;
    const int valid = cols - c;
    if (s.type == MTTKRP_F32) {
        float* p = static_cast<float*>(s.data) + at;
        if (s.whole && valid >= 8) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < valid) p[e] = v[e];
        }
        return;
    }
    uint32_t w[4];
    const bool bf16 = s.type == MTTKRP_BF16;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pair16(bf16, v[2 * e], v[2 * e + 1]);
    uint16_t* p = static_cast<uint16_t*>(s.data) + at;
    if (s.whole && valid >= 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
    }
}

// eight scaled values as hi and lo
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __half2 p = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
        const float2 f = __half22float2(p);
        const __half2 q = __floats2half2_rn(v[2 * e] - f.x, v[2 * e + 1] - f.y);
        h[e] = *reinterpret_cast<const uint32_t*>(&p);
        l[e] = *reinterpret_cast<const uint32_t*>(&q);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void join8(const uint4& hi, const uint4& lo, float* v) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&l[e]));
        v[2 * e] = a.x + b.x;
        v[2 * e + 1] = a.y + b.y;
    }
}

// Sums in tensor memory are cut off towards zero at each addition while they grow to their size.
// What one is short of, as a share of it, after n additions of equal parts: 1.4e-7 for four
// (measured on S X and S S X of 256 x 64: 2.8e-7 and 5.5e-7 short of the exact ones, all of it along the
// result), else by n + 1.
__host__ __device__ constexpr float short_of(int n) { return 0x1.2p-23f / 5.f * (float)(n + 1); }

// That put back, where the sum's last three bits show that it was rounded at all, so that sums of
// few bits stay exact.  An average, found by measurement: sums whose parts are of one sign (the diagonals of S and
// S S) lose it; those of P X, of mixed signs, in which the diagonal's term leads from wherever it lies on, lose
// 0.6 of it.  One step of P X of normal numbers, quintic, along the result: 0.7e-7 (64 x 64) to 1.6e-7 (129 x 130)
// short without, 0.4e-7 to 0.9e-7 too large with it.  Whole errors of five steps against those of fp32 products, 17
// shapes from 20 x 128 to 2048 x 700 and three mixes of strong and weak directions: 0.5 to 1.64 times with it
// everywhere, up to 1.9 without it in P X (64 x 6000), up to 2.35 without it in newton.cu.  With 0.6 of it in P X
// 3 per cent less, but 1.45 instead of 0.98 for 20 x 128.
__device__ __forceinline__ float uncut(float v, float share) {
    return (__float_as_uint(v) & 7u) != 0u ? fmaf(v, share, v) : v;
}

// byte offset of 16-byte piece c (0-7) of row r in a tile
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

struct Source {
    Store g, m, out;            // m.data NULL: no momentum
    uint32_t first[2];          // number of the element's first work item: sums, images
    int slices;                 // sums of a matrix
    int at;                     // number of its first sum
};

// the last of n increasing numbers that is not above x
template <typename F>
__device__ __forceinline__ int element_of(int n, uint32_t x, F first) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first(mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Eight elements each of the gradient and, where there is one, the momentum, of kN places: first what is in
// memory, all of it in flight, then U and what the momentum becomes.  place(i, r, c): whether there is
// an i-th place, and its row and column.  kMomentum: whether there may be one.
template <int kN, bool kMomentum = true>
struct Raws {
    Raw8 g[kN], m[kMomentum ? kN : 1];
    template <typename F>
    __device__ __forceinline__ void get(const Source& s, int b, int cols, F place) {
        const bool momentum = kMomentum && s.m.data != nullptr;
        if (s.g.whole && (!momentum || s.m.whole) && cols % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                int r = 0, c = 0;
                const bool in = place(i, r, c);
                g[i] = raw_fast(s.g, in, b, r, c);
                if constexpr (kMomentum) m[i] = raw_fast(s.m, in && momentum, b, r, c);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                int r = 0, c = 0;
                const bool in = place(i, r, c);
                g[i] = raw_any(s.g, in, b, r, c, cols);
                if (kMomentum && momentum) m[kMomentum ? i : 0] = raw_any(s.m, in, b, r, c, cols);
            }
        }
    }
    __device__ __forceinline__ void update(float mu, bool nesterov, const Source& s, int i, float* u, float* kept) const {
        values(s.g.type, g[i], u);
        if (kMomentum && s.m.data != nullptr) {
            values(s.m.type, m[kMomentum ? i : 0], kept);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kept[e] = fmaf(mu, kept[e], u[e]);
                u[e] = nesterov ? fmaf(mu, kept[e], u[e]) : kept[e];
            }
        }
    }
};

// factors whose product is 2^12 / (|U| + eps); two, as one may leave fp32's range.  Zeros stay zeros, whatever
// eps: 0 / 0 is taken as 0 (squares that leave fp32's range are in the sum's fp64 part, so that only a U of zeros
// has the sum 0).
__device__ __forceinline__ float2 factors(const Sum& total, double eps) {
    const float square = total.hi + total.lo;
    if (square == 0.f && total.wide == 0.0) return make_float2(0.f, 0.f);
    if (total.wide == 0.0 && square >= 0x1p-100f && square <= 0x1p100f)
        return make_float2(1.f, kScale / (sqrtf(square) + (float)eps));
    const double f = (double)kScale / (sqrt((double)total.hi + (double)total.lo + total.wide) + eps);
    const double by = f > 0x1p60 ? 0x1p100 : f < 0x1p-60 ? 0x1p-100 : 1.0;
    return make_float2((float)by, (float)(f / by));
}

struct Result {
    Store out, w;               // w.data NULL: alpha is not used
    float beta;
};

// A warp's stage: 32 rows of kC columns (16 or 32) of fp32, 16-byte pieces in an order in which
// neither rows nor columns meet in a bank.
template <int kC>
__device__ __forceinline__ uint32_t staged(int r, int q) {
    return kC == 32 ? piece(r, q) : (uint32_t)(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}

// one element, and four, of a type of 32 bits or of either of 16
__device__ __forceinline__ float get1(float x, bool) { return x; }
__device__ __forceinline__ float get1(uint16_t x, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ void put1(float* p, bool, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, bool bf16, float v) {
    *p = bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ void get4(const uint4& x, bool, float* v) {
    v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void get4(const uint2& x, bool bf16, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
    v[0] = bf16 ? __uint_as_float(x.x << 16) : f.x, v[1] = bf16 ? __uint_as_float(x.x & 0xFFFF0000u) : f.y;
    v[2] = bf16 ? __uint_as_float(x.y << 16) : g.x, v[3] = bf16 ? __uint_as_float(x.y & 0xFFFF0000u) : g.y;
}
__device__ __forceinline__ void put4(uint4* p, bool, const float* v) {
    *p = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void put4(uint2* p, bool bf16, const float* v) {
    *p = make_uint2(pair16(bf16, v[0], v[1]), pair16(bf16, v[2], v[3]));
}

// Writes them (beta O(U)) to a result, after adding alpha W: whole rows of the stage at a time, or
// where rows are not aligned a column a lane, the old values of kAtOnce rows in flight.  (Four: 64 bf16
// steps of 501 x 333 take 463 us, one row at a time 576; but the registers cost newton_small.cu's
// kernels 3 us whatever they write: one there.)
// (T: float, or uint16_t for either type of 16 bits; kBf16: that it is bf16)
template <typename T, int kC, int kAtOnce, bool kBf16>
__device__ __forceinline__ void write_rows_of(float alpha, const Result& o, int b, int row0, int col0, int rows,
                                              int cols, const uint8_t* stage, int lane) {
    const bool bf16 = kBf16 || o.out.type == MTTKRP_BF16;
    T* const out = static_cast<T*>(o.out.data) + b * o.out.batch;
    const T* const old = o.w.data != nullptr ? static_cast<const T*>(o.w.data) + b * o.w.batch : nullptr;
    if (o.out.whole && (old == nullptr || o.w.whole) && col0 + kC <= cols) {
        using B = typename Bits<4 * sizeof(T)>::type;
        constexpr int kLanes = kC / 4, kStep = 32 / kLanes;
        const int q = lane % kLanes, col = col0 + 4 * q;
        B had[kLanes];
        if (old != nullptr) {
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const int row = row0 + kStep * i + lane / kLanes;
                if (row < rows) had[i] = *reinterpret_cast<const B*>(old + row * o.w.row + col);
            }
        }
#pragma unroll
        for (int i = 0; i < kLanes; ++i) {
            const int r = kStep * i + lane / kLanes, row = row0 + r;
            if (row >= rows) continue;
            const float4 f = *reinterpret_cast<const float4*>(stage + staged<kC>(r, q));
            float v[4] = {f.x, f.y, f.z, f.w};
            if (old != nullptr) {
                float w[4];
                get4(had[i], bf16, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fmaf(alpha, w[e], v[e]);
            }
            put4(reinterpret_cast<B*>(out + row * o.out.row + col), bf16, v);
        }
    } else {
        const int c = lane % kC, col = col0 + c;
        if (col >= cols) return;
        if constexpr (kAtOnce == 1) {
#pragma unroll 4
            for (int r = lane / kC; r < 32; r += 32 / kC) {
                if (row0 + r >= rows) break;
                float v = *reinterpret_cast<const float*>(stage + staged<kC>(r, c >> 2) + (c & 3) * 4);
                const int64_t row = row0 + r;
                if (old != nullptr) v = fmaf(alpha, get1(old[row * o.w.row + col], bf16), v);
                put1(out + row * o.out.row + col, bf16, v);
            }
        } else {
            constexpr int kStep = 32 / kC;
            const int first = lane / kC, n = rows - row0 < 32 ? rows - row0 : 32;
            T* to = out + (row0 + first) * o.out.row + col;
            const T* from = old != nullptr ? old + (row0 + first) * o.w.row + col : nullptr;
#pragma unroll 1
            for (int r0 = first; r0 < n; r0 += kAtOnce * kStep) {
                T had[kAtOnce];
                float v[kAtOnce];
                if (old != nullptr) {
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        if (r0 + i * kStep < n) had[i] = *from;
                        from += kStep * o.w.row;
                    }
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)       // (the stage has 32 rows)
                    v[i] = *reinterpret_cast<const float*>(stage + staged<kC>((r0 + i * kStep) & 31, c >> 2) + (c & 3) * 4);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    if (old != nullptr) v[i] = fmaf(alpha, get1(had[i], bf16), v[i]);
                    if (r0 + i * kStep < n) put1(to, bf16, v[i]);
                    to += kStep * o.out.row;
                }
            }
        }
    }
}
template <int kC, int kAtOnce, bool kBf16 = false>
__device__ __forceinline__ void write_rows(float alpha, const Result& o, int b, int row0, int col0, int rows,
                                           int cols, const uint8_t* stage, int lane) {
    if (!kBf16 && o.out.type == MTTKRP_F32)
        write_rows_of<float, kC, kAtOnce, false>(alpha, o, b, row0, col0, rows, cols, stage, lane);
    else
        write_rows_of<uint16_t, kC, kAtOnce, kBf16>(alpha, o, b, row0, col0, rows, cols, stage, lane);
}

// ---- host

// the matrices of m from number b0 on
inline Store store_of(const mttkrp_matrices& m, int64_t b0) {
    const int64_t elem = m.type == MTTKRP_F32 ? 4 : 2, row = m.rows > 1 ? m.row_stride : 0, batch = m.batch > 1 ? m.batch_stride : 0;
    Store s;
    s.data = static_cast<uint8_t*>(m.data) + b0 * batch * elem;
    s.row = row;
    s.batch = batch;
    s.type = (uint8_t)m.type;
    s.whole = (reinterpret_cast<uintptr_t>(m.data) % 16 == 0 && row * elem % 16 == 0 && batch * elem % 16 == 0) ? 1 : 0;
    return s;
}

// A launch of clusters whose start overlaps the end of the kernel before it (see launch.cuh).
template <typename K, typename A> cudaError_t launch_clusters(K kernel, unsigned blocks, unsigned threads, size_t smem, int cluster, cudaStream_t s, const A& args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(blocks);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    config.attrs = attr;
    config.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&config, kernel, args);
    if (e != cudaSuccess) cudaGetLastError();       // the error is told by this call alone
    return e;
}

}  // namespace mk
