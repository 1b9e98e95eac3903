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
// come as turns a position in 64-bit fixed point instead, within half a unit (turns.h); the
// product's low 64 bits are the angle as a fraction of a turn, within |p| 2^-65 of one (2e-7
// radians at 2^40), and a negative position turns back.  Its nearest quarter is taken off as an
// integer, so that what fp32 rounds, three times, is at most an eighth of a turn (1.2e-7 radians).
#include <algorithm>
#include <atomic>

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

// Dense tensors whose rows start at any element.  A CTA takes some rows, which lie in one piece of
// memory: loads and stores are whole aligned 16-byte vectors of it (its ends element by element), and
// the rows are turned in shared memory at the same offset.  What bounds it is the wait for the loads
// of a CTA, which nothing of its own covers: 24 KB a CTA keep eight of them on a multiprocessor.
// (84M bf16 in rows of 171: 24 heads 76 us, element by element from memory 77 in halves and 140 for
// neighbours; 10 heads 78, 113 and 137 in rows of 83; one head 171, 286 and 209.)
constexpr int kStageBytes = 24576;      // of rows, at most, but for one token that takes more
constexpr int kMostStage = 98304;
constexpr int kMostShared = kMostStage + 32;    // a piece of that at any offset, in whole vectors
constexpr int kFewest = 608;            // CTAs before they take more than one token: four a multiprocessor

struct Dense {
    const void* x;
    void* y;
    uint64_t rows;                      // all of them: fewer than 2^32
    uint32_t per_cta;                   // rows: whole tokens where heads follow one another
    uint32_t heads;                     // rows in a token that follow one another, or 1
    uint32_t outside;                   // else heads that lie outside of the tokens
};

template <int kPairs>
struct DenseArgs {
    Dense t[kMaxTensors];
    const void* positions;
    int64_t pb, pt;
    uint32_t length;
    int dims, half, width;
    float scale;
    bool wide, inverse;
    uint64_t turns[kPairs];
};

template <typename T, bool kNeighbours, int kPairs>
__global__ void __launch_bounds__(kThreads) dense_kernel(const __grid_constant__ DenseArgs<kPairs> a) {
    extern __shared__ __align__(16) uint8_t room[];
    after_previous();
    const Dense d = a.t[blockIdx.y];
    const uint64_t row0 = (uint64_t)blockIdx.x * d.per_cta;
    if (row0 >= d.rows) return;
    const uint32_t rows = (uint32_t)min(d.rows - row0, (uint64_t)d.per_cta);
    const T* const from = static_cast<const T*>(d.x) + row0 * a.width;
    T* const to = static_cast<T*>(d.y) + row0 * a.width;
    constexpr uint32_t kVec = 16 / sizeof(T);
    // elements before the first one in its vector; vectors that are whole
    const uint32_t shift = (uint32_t)((reinterpret_cast<uintptr_t>(from) & 15) / sizeof(T)), n = rows * (uint32_t)a.width;
    T* const s = reinterpret_cast<T*>(room) + shift;
    const uint32_t v0 = shift == 0 ? 0 : 1, v1 = (shift + n) / kVec;
    const uint32_t head = v1 >= v0 && v0 * kVec >= shift ? min(v0 * kVec - shift, n) : n;      // elements before the first whole one
    const uint32_t tail = v1 > v0 ? v1 * kVec - shift : head;                                   // first one behind the last
    for (uint32_t v = v0 + threadIdx.x; v < v1; v += kThreads)
        reinterpret_cast<uint4*>(room)[v] = __ldcs(reinterpret_cast<const uint4*>(from - shift) + v);
    for (uint32_t e = threadIdx.x; e < head; e += kThreads) s[e] = from[e];
    for (uint32_t e = tail + threadIdx.x; e < n; e += kThreads) s[e] = from[e];
    __syncthreads();
    // a thread's pairs: number i of a token's rows
    const uint32_t tokens = rows / d.heads, first = (uint32_t)row0 / d.heads;
    uint32_t token = threadIdx.x / (uint32_t)a.half, i = threadIdx.x - token * (uint32_t)a.half;
    const uint32_t token_step = kThreads / (uint32_t)a.half, i_step = kThreads - token_step * (uint32_t)a.half;
    const uint64_t* turns = a.turns;
    asm volatile("" : "+l"(turns));         // (see Unit::frequencies)
    while (token < tokens) {
        const uint32_t at = first + token, group = at / a.length, t = at - group * a.length;
        const uint32_t b = d.outside > 0 ? group / d.outside : group;
        const int64_t where = (int64_t)b * a.pb + (int64_t)t * a.pt;
        uint64_t p = a.wide ? (uint64_t)static_cast<const int64_t*>(a.positions)[where]
                            : (uint64_t)(int64_t)static_cast<const int32_t*>(a.positions)[where];
        if (a.inverse) p = 0 - p;
        float c, sn;
        cos_sin(p * turns[i], a.scale, c, sn);
        T* u = s + token * d.heads * (uint32_t)a.width + (kNeighbours ? 2 * i : i);
        const int other = kNeighbours ? 1 : a.half;
#pragma unroll 4
        for (uint32_t h = 0; h < d.heads; ++h, u += a.width) {
            const float m = to_f32(u[0]), q = to_f32(u[other]);
            u[0] = from_f32<T>(m * c - q * sn);
            u[other] = from_f32<T>(m * sn + q * c);
        }
        token += token_step;
        i += i_step;
        if (i >= (uint32_t)a.half) {
            i -= (uint32_t)a.half;
            ++token;
        }
    }
    __syncthreads();
    for (uint32_t v = v0 + threadIdx.x; v < v1; v += kThreads)
        __stcs(reinterpret_cast<uint4*>(to - shift) + v, reinterpret_cast<const uint4*>(room)[v]);
    for (uint32_t e = threadIdx.x; e < head; e += kThreads) to[e] = s[e];
    for (uint32_t e = tail + threadIdx.x; e < n; e += kThreads) to[e] = s[e];
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

// Whether the rows of a tensor and of its result fill their memory in the order of tokens and heads
// (heads = 0) or of heads and tokens in every batch (their number in `outside`), at the same offset from
// 16 bytes.
bool dense(const RotaryArgs& r, const mttkrp_rotary_tensor& t, Dense& d) {
    const int64_t w = r.width, h = t.heads, n = r.length;
    auto is = [&](const int64_t* s, int64_t batch, int64_t token, int64_t head) {
        return (r.batch == 1 || s[0] == batch) && (n == 1 || s[1] == token) && (h == 1 || s[2] == head);
    };
    if (((reinterpret_cast<uintptr_t>(t.x) ^ reinterpret_cast<uintptr_t>(t.out)) & 15) != 0) return false;
    d.x = t.x;
    d.y = t.out;
    d.rows = (uint64_t)r.batch * n * h;
    if (is(t.x_strides, n * h * w, h * w, w) && is(t.out_strides, n * h * w, h * w, w)) {
        d.heads = (uint32_t)h;
        d.outside = 0;
    } else if (is(t.x_strides, n * h * w, w, n * w) && is(t.out_strides, n * h * w, w, n * w)) {
        d.heads = 1;
        d.outside = (uint32_t)h;
    } else {
        return false;
    }
    return true;
}

// Allows a form of the kernel what any call may take, once a device: the limit is the function's own, and
// another thread's call may lie between the one here and the launch.
template <typename T, bool kNeighbours, int kPairs>
cudaError_t allow() {
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && allowed[dev])) return e;
    e = cudaFuncSetAttribute(dense_kernel<T, kNeighbours, kPairs>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e == cudaSuccess && dev < 64) allowed[dev] = true;
    return e;
}

template <typename T, int kPairs>
cudaError_t run_dense(const RotaryArgs& r, cudaStream_t s, bool& taken) {
    DenseArgs<kPairs> a;
    uint64_t blocks = 0;
    size_t most = 0;
    taken = false;
    for (int k = 0; k < r.n; ++k) {
        Dense& d = a.t[k];
        if (!dense(r, r.tensor[k], d)) return cudaSuccess;
        if (d.rows > UINT32_MAX || d.heads * (uint64_t)r.width > kMostStage / sizeof(T)) return cudaSuccess;
        const size_t token = (size_t)d.heads * r.width * sizeof(T);
        const uint64_t spread = d.rows / d.heads / kFewest;         // tokens
        d.per_cta = d.heads * (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(kStageBytes / token, spread));
        most = std::max(most, (size_t)d.per_cta * r.width * sizeof(T));
        blocks = std::max(blocks, (d.rows + d.per_cta - 1) / d.per_cta);
    }
    if (blocks > INT32_MAX) return cudaSuccess;
    a.positions = r.positions;
    a.pb = r.pos_batch_stride;
    a.pt = r.pos_stride;
    a.length = (uint32_t)r.length;
    a.dims = r.dims;
    a.half = r.dims / 2;
    a.width = (int)r.width;
    a.scale = r.scale;
    a.wide = r.pos_bytes == 8;
    a.inverse = r.inverse;
    for (int i = 0; i < r.dims / 2; ++i) a.turns[i] = r.turns[i];
    taken = true;
    const size_t smem = (most + 15 + 16) / 16 * 16;     // and up to a vector before the first element
    const cudaError_t e = r.interleaved ? allow<T, true, kPairs>() : allow<T, false, kPairs>();
    if (e != cudaSuccess) return e;
    const auto kernel = r.interleaved ? dense_kernel<T, true, kPairs> : dense_kernel<T, false, kPairs>;
    return launch_early(kernel, dim3((unsigned)blocks, (unsigned)r.n), kThreads, smem, s, a);
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
    // (fp32 in halves, 24 heads: 114 us element by element from memory, 130 through shared memory;
    // one head: 284 and 188)
    if (v == 1 && (sizeof(T) == 2 || r.interleaved || a.heads < kRows)) {
        bool taken;
        const cudaError_t e = run_dense<T, kPairs>(r, s, taken);
        if (taken) return e;
    }
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
