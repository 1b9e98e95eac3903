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
// at most an eighth of a turn (4.7e-8 radians).
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

// cos and sin of `phase` 2^-64 turns, by the Taylor series up to an eighth of a turn either
// way (the first terms left out: 2e-9 and 1e-10)
__device__ __forceinline__ void cos_sin(uint64_t phase, float scale, float& c, float& s) {
    const uint32_t at = (uint32_t)(phase >> 32);
    const uint32_t quarter = (at + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(at - (quarter << 30));          // in [-2^29, 2^29)
    const float x = (float)rest * 1.4629180792671596e-9f;          // 2 pi 2^-32
    const float z = x * x;
    float u = fmaf(z, 1.f / 362880.f, -1.f / 5040.f), v = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    u = fmaf(z, u, 1.f / 120.f);
    v = fmaf(z, v, -1.f / 720.f);
    u = fmaf(z, u, -1.f / 6.f);
    v = fmaf(z, v, 1.f / 24.f);
    u = fmaf(x * z, u, x);                                          // sine
    v = fmaf(z, fmaf(z, v, -0.5f), 1.f);                            // cosine
    c = (quarter & 1 ? u : v) * scale;
    s = (quarter & 1 ? v : u) * scale;
    c = __uint_as_float(__float_as_uint(c) ^ (((quarter + 1) & 2) << 30));      // quarters 1 and 2
    s = __uint_as_float(__float_as_uint(s) ^ ((quarter & 2) << 30));            // quarters 2 and 3
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

// What a thread of a launch works on, from its number: a vector (or pair of vectors) of a row.
template <int kPairs>
struct Place {
    uint64_t row;           // token, or token and head
    uint32_t b, t;
    int unit, column, valid;
    bool turns;
};

template <int V, int kPairs>
__device__ __forceinline__ void columns(const Args<kPairs>& a, Place<kPairs>& p) {
    p.turns = p.unit < a.units;
    p.column = p.turns ? p.unit * V : a.dims + (p.unit - a.units) * V;
    p.valid = a.width - p.column;
}

template <int kPairs>
__device__ __forceinline__ uint64_t position(const Args<kPairs>& a, uint32_t b, uint32_t t) {
    const int64_t where = (int64_t)b * a.pb + (int64_t)t * a.pt;
    const uint64_t p = a.wide ? (uint64_t)static_cast<const int64_t*>(a.positions)[where]
                              : (uint64_t)(int64_t)static_cast<const int32_t*>(a.positions)[where];
    return a.inverse ? 0 - p : p;
}

// What a thread turns at once: two vectors `half` columns apart, whose elements are pairs
// (kHalves) or hold neighbours that are (kSplit), or one vector of neighbours (kSingle, where
// half of the columns is no multiple of a vector).
enum Layout { kHalves, kSplit, kSingle };

template <typename T, int V, bool kWhole, Layout kLayout>
struct Unit {
    static constexpr int kVecs = kLayout == kSingle ? 1 : 2;
    static constexpr int kAngles = kVecs * V / 2;
    static_assert(kLayout == kHalves || V >= 2, "a pair of neighbours in a vector");
    Pack<T, V> v[kVecs];
    __device__ __forceinline__ void get(const T* p, int half, int valid, bool turns) {
        v[0] = load<T, V, kWhole>(p, valid);
        if (kVecs == 2 && turns) v[kVecs - 1] = load<T, V, kWhole>(p + half, valid);
    }
    __device__ __forceinline__ void put(T* p, int half, int valid, bool turns) const {
        store<T, V, kWhole>(p, v[0], valid);
        if (kVecs == 2 && turns) store<T, V, kWhole>(p + half, v[kVecs - 1], valid);
    }
    __device__ __forceinline__ void turn(int e, float c, float s) {
        T& p = kLayout == kHalves ? v[0].v[e] : v[2 * e / V].v[2 * e % V];
        T& q = kLayout == kHalves ? v[kVecs - 1].v[e] : v[2 * e / V].v[2 * e % V + 1];
        const float m = to_f32(p), n = to_f32(q);
        p = from_f32<T>(m * c - n * s);
        q = from_f32<T>(m * s + n * c);
    }
    // Its frequencies.  By a plain load: lanes read different ones, which the path of constants
    // (where arguments lie) would serve one after the other (200003 rows of 256 fp32: 215 us, 96 so).
    template <int kPairs>
    __device__ __forceinline__ static void frequencies(const Args<kPairs>& a, int unit, uint64_t* f) {
        constexpr int kFirst = kLayout == kSplit ? kAngles / 2 : kAngles;
        const uint64_t* at = a.turns + unit * kFirst;
        asm volatile("" : "+l"(at));
#pragma unroll
        for (int e = 0; e < kAngles; ++e) f[e] = e < kFirst ? at[e] : at[a.half / 2 + e - kFirst];
    }
};

// A thread keeps the angles of its token and walks heads.
template <typename T, int V, bool kWhole, Layout kLayout, int kPairs>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ Args<kPairs> a) {
    after_previous();
    using U = Unit<T, V, kWhole, kLayout>;
    Place<kPairs> p;
    const uint32_t per = (uint32_t)(a.units + a.copies);
    const uint64_t at = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    if (a.few) {
        p.row = (uint32_t)at / per;
        p.b = (uint32_t)p.row / a.length;
    } else {
        p.row = at / per;
        p.b = (uint32_t)(p.row / a.length);
    }
    if (p.row >= a.tokens) return;
    p.unit = (int)(at - p.row * per);
    p.t = (uint32_t)(p.row - (uint64_t)p.b * a.length);
    columns<V>(a, p);
    float c[U::kAngles], s[U::kAngles];
    const int h0 = blockIdx.y * a.chunk, h1 = h0 + a.chunk < a.heads ? h0 + a.chunk : a.heads;
    bool angles = p.turns;      // still to be worked out, behind the first loads
    int k = 0;
    for (int h = h0; h < h1;) {
        while (k + 1 < a.n && a.t[k + 1].first <= h) ++k;
        const Tensor& x = a.t[k];
        const int end = k + 1 < a.n && a.t[k + 1].first < h1 ? a.t[k + 1].first : h1;
        if (!p.turns && x.same) {
            h = end;
            continue;
        }
        const T* from = static_cast<const T*>(x.x) + p.b * x.xb + p.t * x.xt + (h - x.first) * x.xh + p.column;
        T* to = static_cast<T*>(x.y) + p.b * x.yb + p.t * x.yt + (h - x.first) * x.yh + p.column;
        for (; h < end; h += kRows, from += kRows * x.xh, to += kRows * x.yh) {
            U u[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (h + r < end) u[r].get(from + r * x.xh, a.half, p.valid, p.turns);
            if (angles) {
                const uint64_t where = position(a, p.b, p.t);
                uint64_t f[U::kAngles];
                U::frequencies(a, p.unit, f);
#pragma unroll
                for (int e = 0; e < U::kAngles; ++e) cos_sin(where * f[e], a.scale, c[e], s[e]);
                angles = false;
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (h + r >= end) break;
                if (p.turns) {
#pragma unroll
                    for (int e = 0; e < U::kAngles; ++e) u[r].turn(e, c[e], s[e]);
                }
                u[r].put(to + r * x.yh, a.half, p.valid, p.turns);
            }
        }
        h = end;
    }
}

// Few heads: a thread takes one unit of kRows rows (each a token and a head of one tensor),
// `step` rows apart, and the angles of each.
template <typename T, int V, bool kWhole, Layout kLayout, int kPairs>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ Args<kPairs> a, uint64_t step) {
    after_previous();
    using U = Unit<T, V, kWhole, kLayout>;
    const uint32_t per = (uint32_t)(a.units + a.copies);
    const uint64_t at = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    Place<kPairs> p;
    p.row = a.few ? (uint64_t)((uint32_t)at / per) : at / per;
    if (p.row >= step) return;
    p.unit = (int)(at - p.row * per);
    columns<V>(a, p);
    const uint64_t rows = a.tokens * (uint32_t)a.heads;
    U u[kRows];
    T* to[kRows];
    uint64_t where[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const uint64_t row = p.row + r * step;
        to[r] = nullptr;        // nothing to do
        where[r] = 0;
        if (row >= rows) continue;
        const uint64_t token = a.few ? (uint64_t)((uint32_t)row / (uint32_t)a.heads) : row / (uint32_t)a.heads;
        const int h = (int)(row - token * (uint32_t)a.heads);
        const uint32_t b = (uint32_t)token / a.length, t = (uint32_t)token - b * a.length;
        int k = 0;
        while (k + 1 < a.n && a.t[k + 1].first <= h) ++k;
        const Tensor& x = a.t[k];
        if (!p.turns && x.same) continue;
        where[r] = position(a, b, t);
        u[r].get(static_cast<const T*>(x.x) + b * x.xb + t * x.xt + (h - x.first) * x.xh + p.column, a.half, p.valid, p.turns);
        to[r] = static_cast<T*>(x.y) + b * x.yb + t * x.yt + (h - x.first) * x.yh + p.column;
    }
    uint64_t f[U::kAngles];
    if (p.turns) U::frequencies(a, p.unit, f);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (to[r] == nullptr) continue;
        if (p.turns) {
#pragma unroll
            for (int e = 0; e < U::kAngles; ++e) {
                float c, s;
                cos_sin(where[r] * f[e], a.scale, c, s);
                u[r].turn(e, c, s);
            }
        }
        u[r].put(to[r], a.half, p.valid, p.turns);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The largest number of elements, a power of two up to 16 bytes, that divides everything a
// vector starts at (half of the columns too, but that neighbours stay together: 2 at least).
int vector_of(const RotaryArgs& r, int elem) {
    const uint64_t half = (uint64_t)r.dims / 2;
    uint64_t all = 16 / elem;
    all |= (uint64_t)r.width | (uint64_t)r.dims | (r.interleaved && half % 2 != 0 ? 2 : half);
    for (int k = 0; k < r.n; ++k) {
        const mttkrp_rotary_tensor& t = r.tensor[k];
        for (int m = 0; m < 3; ++m) all |= (uint64_t)t.x_strides[m] | (uint64_t)t.out_strides[m];
        all |= (uint64_t)((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.out)) / elem);
    }
    return (int)(all & (0 - all));
}

template <typename T, int V, bool kWhole, Layout kLayout, int kPairs>
cudaError_t launch(Args<kPairs>& a, cudaStream_t s) {
    const uint64_t per = (uint64_t)(a.units + a.copies);
    if (a.heads < kRows) {
        const uint64_t rows = a.tokens * a.heads;
        const uint64_t step = rows * per < kEnough ? rows : (rows + kRows - 1) / kRows;
        const uint64_t blocks = (step * per + kThreads - 1) / kThreads;
        if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
        a.few = step * per < (uint64_t)UINT32_MAX - kThreads && rows <= UINT32_MAX;
        return launch_early(rows_kernel<T, V, kWhole, kLayout, kPairs>, dim3((unsigned)blocks), kThreads, 0, s, a, step);
    }
    const uint64_t threads = a.tokens * per, blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    a.few = threads < (uint64_t)UINT32_MAX - kThreads;
    a.chunk = a.heads;
    while (a.chunk > 1 && threads * cdiv(a.heads, a.chunk) < kEnough) a.chunk = (a.chunk + 1) / 2;
    if (a.chunk > kRows) a.chunk = (int)cdiv(a.chunk, kRows) * kRows;       // whole groups of loads
    a.chunk = std::max(a.chunk, (int)cdiv(a.heads, 65535));     // the grid's second dimension
    const unsigned chunks = (unsigned)cdiv(a.heads, a.chunk);
    return launch_early(heads_kernel<T, V, kWhole, kLayout, kPairs>, dim3((unsigned)blocks, chunks), kThreads, 0, s, a);
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
    const int v = vector_of(r, sizeof(T)), half = r.dims / 2;
    if (!r.interleaved) {
        a.units = half / v;
        a.copies = copies ? (a.width - r.dims) / v : 0;
        if (v == 1) return launch<T, 1, true, kHalves>(a, s);
        if (v == 2) return launch<T, 2, true, kHalves>(a, s);
        if constexpr (sizeof(T) == 2)
            if (v == 8) return launch<T, 8, true, kHalves>(a, s);
        return launch<T, 4, true, kHalves>(a, s);
    }
    // neighbours at any offset are read element by element
    const int step = v < 2 ? 2 : v;
    a.units = half % 2 == 0 ? half / step : half;
    a.copies = copies ? (int)cdiv(a.width - r.dims, step) : 0;
    if (half % 2 != 0) return v < 2 ? launch<T, 2, false, kSingle>(a, s) : launch<T, 2, true, kSingle>(a, s);
    if (v < 2) return launch<T, 2, false, kSplit>(a, s);
    if (v == 2) return launch<T, 2, true, kSplit>(a, s);
    if constexpr (sizeof(T) == 2)
        if (v == 8) return launch<T, 8, true, kSplit>(a, s);
    return launch<T, 4, true, kSplit>(a, s);
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
