// Rows rotated by their position: for pair i of the first `dims` columns of a row at
// position p, with the angle a = p f_i,
//   u' = s (u cos a - v sin a),   v' = s (u sin a + v cos a);
// the columns behind are copied.  The gradient is the rotation by -a.
//
// Bound by memory: one read and one write of every element.  A thread holds the cosines
// and sines of one vector's pairs and walks heads of all tensors of one token, so an
// angle is worked out once for as many heads as a thread takes, four rows' loads in flight.
// Heads are dealt out to as many threads as fill the GPU (few tokens: a head each).
//
// The angle.  p f_i in fp32 is off by p f_i 2^-24: 0.06 radians at a million.  Frequencies
// come as turns a position in 64-bit fixed point instead; the product's low 64 bits are
// the angle as a fraction of a turn, exact however far the position, and a negative one
// turns back.  Its nearest quarter is taken off as an integer, so that what fp32 rounds is
// at most an eighth of a turn (2.3e-8 radians), and sincospi does the rest.
#include <algorithm>

#include "launch.cuh"
#include "rotary.h"
#include "types.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTensors = MTTKRP_MAX_ROTARY;
constexpr int kRows = 4;            // rows a thread has in flight
constexpr uint64_t kEnough = 600000;    // threads that fill the GPU twice

struct Tensor {
    const void* x;
    void* y;
    int64_t xb, xt, xh, yb, yt, yh;     // strides in elements: batch, token, head
    int first;                          // heads of the tensors before it
    bool same;                          // y is x: nothing to copy
};

template <int kPairs>
struct Args {
    Tensor t[kMaxTensors];
    const void* positions;
    int64_t pb, pt;
    uint64_t tokens;                    // batch * length
    uint32_t length;
    int n, heads, chunk;                // heads of all tensors; heads a thread takes
    int units, copies;                  // vectors a row that are rotated (pairs of vectors of halves), copied
    int dims, half, width;
    float scale;
    bool wide, inverse, few;            // wide: 64-bit positions; few: vectors of all tokens below 2^32
    uint64_t turns[kPairs];
};

// cos and sin of `phase` 2^-64 turns
__device__ __forceinline__ void cos_sin(uint64_t phase, float scale, float& c, float& s) {
    const uint32_t at = (uint32_t)(phase >> 32);
    const uint32_t quarter = (at + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(at - (quarter << 30));          // in [-2^29, 2^29)
    float x, y;
    sincospif((float)rest * 0x1p-31f, &y, &x);
    c = quarter & 1 ? y : x;
    s = quarter & 1 ? x : y;
    c = ((quarter + 1) & 2 ? -c : c) * scale;                       // quarters 1 and 2
    s = (quarter & 2 ? -s : s) * scale;                             // quarters 2 and 3
}

// V elements at p; kWhole: p is aligned to all of them, else the first n of them
template <typename T, int V, bool kWhole>
__device__ __forceinline__ Pack<T, V> load(const T* p, int n) {
    Pack<T, V> v;
    if constexpr (kWhole) {
        v = as_pack<Pack<T, V>>(__ldcs(reinterpret_cast<const typename Bits<V * sizeof(T)>::type*>(p)));
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e == 0 || e < n) v.v[e] = p[e];
    }
    return v;
}

template <typename T, int V, bool kWhole>
__device__ __forceinline__ void store(T* p, const Pack<T, V>& v, int n) {
    if constexpr (kWhole) {
        __stcs(reinterpret_cast<typename Bits<V * sizeof(T)>::type*>(p), as_pack<typename Bits<V * sizeof(T)>::type>(v));
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e == 0 || e < n) p[e] = v.v[e];
    }
}

// kTogether: a pair's columns are neighbours (a unit is one vector), else `half` apart (a
// unit is two vectors)
template <typename T, int V, bool kWhole, bool kTogether, int kPairs>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args<kPairs> a) {
    after_previous();
    constexpr int kAngles = kTogether ? V / 2 : V;
    using P = Pack<T, V>;
    const uint32_t per = (uint32_t)(a.units + a.copies);
    const uint64_t at = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    uint64_t token;
    uint32_t b;
    if (a.few) {
        token = (uint32_t)at / per;
        b = (uint32_t)token / a.length;
    } else {
        token = at / per;
        b = (uint32_t)(token / a.length);
    }
    if (token >= a.tokens) return;
    const int unit = (int)(at - token * per);
    const uint32_t t = (uint32_t)(token - (uint64_t)b * a.length);
    const bool turns = unit < a.units;
    const int column = turns ? unit * V : a.dims + (unit - a.units) * V;
    const int valid = a.width - column;
    float c[kAngles], s[kAngles];
    if (turns) {
        const int64_t where = (int64_t)b * a.pb + (int64_t)t * a.pt;
        uint64_t p = a.wide ? (uint64_t)static_cast<const int64_t*>(a.positions)[where]
                            : (uint64_t)(int64_t)static_cast<const int32_t*>(a.positions)[where];
        if (a.inverse) p = 0 - p;
#pragma unroll
        for (int e = 0; e < kAngles; ++e) cos_sin(p * a.turns[unit * kAngles + e], a.scale, c[e], s[e]);
    }
    const int h0 = blockIdx.y * a.chunk, h1 = h0 + a.chunk < a.heads ? h0 + a.chunk : a.heads;
    int k = 0;
    for (int h = h0; h < h1;) {
        while (k + 1 < a.n && a.t[k + 1].first <= h) ++k;
        const Tensor& x = a.t[k];
        const int end = k + 1 < a.n && a.t[k + 1].first < h1 ? a.t[k + 1].first : h1;
        const T* from = static_cast<const T*>(x.x) + (int64_t)b * x.xb + (int64_t)t * x.xt + (int64_t)(h - x.first) * x.xh + column;
        T* to = static_cast<T*>(x.y) + (int64_t)b * x.yb + (int64_t)t * x.yt + (int64_t)(h - x.first) * x.yh + column;
        if (!turns && x.same) {
            h = end;
            continue;
        }
        for (; h < end; h += kRows, from += kRows * x.xh, to += kRows * x.yh) {
            P u[kRows], v[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (h + r >= end) break;
                u[r] = load<T, V, kWhole>(from + r * x.xh, valid);
                if (!kTogether && turns) v[r] = load<T, V, kWhole>(from + r * x.xh + a.half, valid);
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (h + r >= end) break;
                if (turns) {
#pragma unroll
                    for (int e = 0; e < kAngles; ++e) {
                        T& p = kTogether ? u[r].v[2 * e] : u[r].v[e];
                        T& q = kTogether ? u[r].v[2 * e + 1] : v[r].v[e];
                        const float m = to_f32(p), n = to_f32(q);
                        p = from_f32<T>(m * c[e] - n * s[e]);
                        q = from_f32<T>(m * s[e] + n * c[e]);
                    }
                    if (!kTogether) store<T, V, kWhole>(to + r * x.yh + a.half, v[r], valid);
                }
                store<T, V, kWhole>(to + r * x.yh, u[r], valid);
            }
        }
        h = end;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// the largest number of elements, a power of two up to 16 bytes, that divides everything a
// vector starts at
int vector_of(const RotaryArgs& r, int elem) {
    uint64_t all = 16 / elem;
    const int64_t half = r.dims / 2;
    all |= (uint64_t)(r.interleaved ? r.dims : half) | (uint64_t)r.dims | (uint64_t)r.width;
    for (int k = 0; k < r.n; ++k) {
        const mttkrp_rotary_tensor& t = r.tensor[k];
        for (int m = 0; m < 3; ++m) all |= (uint64_t)t.x_strides[m] | (uint64_t)t.out_strides[m];
        all |= (uint64_t)((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.out)) / elem);
    }
    return (int)(all & (0 - all));
}

template <typename T, int V, bool kWhole, bool kTogether, int kPairs>
cudaError_t launch(const Args<kPairs>& a, uint64_t blocks, cudaStream_t s) {
    const unsigned chunks = (unsigned)cdiv(a.heads, a.chunk);
    return launch_early(rotary_kernel<T, V, kWhole, kTogether, kPairs>, dim3((unsigned)blocks, chunks), kThreads, 0, s, a);
}

template <typename T, int kPairs>
cudaError_t run(const RotaryArgs& r, cudaStream_t s) {
    Args<kPairs> a;
    a.n = r.n;
    a.heads = 0;
    bool copies = false;
    for (int k = 0; k < r.n; ++k) {
        const mttkrp_rotary_tensor& t = r.tensor[k];
        const bool same = t.x == t.out;
        a.t[k] = Tensor{t.x, t.out, t.x_strides[0], t.x_strides[1], t.x_strides[2],
                        t.out_strides[0], t.out_strides[1], t.out_strides[2], a.heads, same};
        a.heads += (int)t.heads;
        copies = copies || !same;
    }
    a.positions = r.positions;
    a.pb = r.pos_batch_stride;
    a.pt = r.pos_stride;
    a.tokens = (uint64_t)r.batch * r.length;
    a.length = (uint32_t)r.length;
    a.dims = r.dims;
    a.half = r.dims / 2;
    a.width = (int)r.width;
    a.scale = r.scale;
    a.wide = r.pos_bytes == 8;
    a.inverse = r.inverse;
    for (int i = 0; i < r.dims / 2; ++i) a.turns[i] = r.turns[i];
    const int v = vector_of(r, sizeof(T));
    const bool pieces = r.interleaved && v < 2;         // a pair of neighbours, element by element
    const int step = pieces ? 2 : v;
    a.units = (r.interleaved ? r.dims : r.dims / 2) / step;
    a.copies = copies ? (int)cdiv(r.width - r.dims, step) : 0;
    const uint64_t threads = a.tokens * (uint64_t)(a.units + a.copies);
    const uint64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    a.few = threads < (uint64_t)UINT32_MAX - kThreads;
    a.chunk = a.heads;
    while (a.chunk > 1 && threads * cdiv(a.heads, a.chunk) < kEnough) a.chunk = (a.chunk + 1) / 2;
    a.chunk = std::max(a.chunk, (int)cdiv(a.heads, 65535));     // the grid's second dimension
    if (r.interleaved) {
        if (pieces) return launch<T, 2, false, true>(a, blocks, s);
        if (v == 2) return launch<T, 2, true, true>(a, blocks, s);
        if constexpr (sizeof(T) == 2)
            if (v == 8) return launch<T, 8, true, true>(a, blocks, s);
        return launch<T, 4, true, true>(a, blocks, s);
    }
    if (v == 1) return launch<T, 1, true, false>(a, blocks, s);
    if (v == 2) return launch<T, 2, true, false>(a, blocks, s);
    if constexpr (sizeof(T) == 2)
        if (v == 8) return launch<T, 8, true, false>(a, blocks, s);
    return launch<T, 4, true, false>(a, blocks, s);
}

template <typename T>
cudaError_t run(const RotaryArgs& r, cudaStream_t s) {
    // 2 and 5 KB of arguments a launch
    return r.dims <= 2 * 128 ? run<T, 128>(r, s) : run<T, MTTKRP_MAX_ROTARY_DIMS / 2>(r, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
    switch (a.type) {
        case MTTKRP_F32: return run<float>(a, s);
        case MTTKRP_BF16: return run<__nv_bfloat16>(a, s);
        default: return run<__half>(a, s);
    }
}

}  // namespace mk
