// Orthogonalisation of matrices of which one side is at most 128, in one launch: a cluster of
// CTAs keeps the matrix in shared memory through all steps.  (The arithmetic and the images are
// those of newton.cu, with both parts of every operand; its launches, 17 for five steps, take
// 90 us for a 256 x 64 matrix, of which next to nothing is work.)
//
// Every CTA holds a slab of X: all of the short side, some tiles of 64 along the long one.
// A step: the slab's part of S = X X^T (every 64 indices from tensor memory into registers); the
// parts added up over the cluster, each CTA some rows, and spread again; P, by every CTA; its
// slab of P X, written over X.  S and P are whole (up to 128 x 128).  What a step costs is mostly
// latency: 33 us for five steps of 256 x 64, 5 us a step; 48 us for 128 x 128.
//
// One CTA an SM whatever the size (the launch asks for most of the shared memory): a second
// one would wait for the tensor memory of the first, which may wait for its cluster.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "launch.cuh"
#include "newton.cuh"
#include "newton.h"

namespace mk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kHeader = 1024;              // barriers, sums, flags
constexpr uint32_t kSmem = 232448 - 512;        // all but what is static: one CTA an SM
constexpr uint32_t kTiles = (kSmem - 1024 - kHeader) / kTileBytes;      // 28
constexpr uint32_t kHalfTmem = 256;             // columns of one of two buffers of accumulators

struct Partial {
    float hi, lo;
    double wide;
};

constexpr int kElements = 64;       // list elements a launch: 14 KB of arguments

struct SmallArgs {
    int n, steps;
    float mu, alpha;
    bool nesterov;
    double eps;
    uint32_t* status;
    Shape shape[kElements];
    Source source[kElements];
    Result result[kElements];
    float abc[3 * kNewtonMaxSteps];
};

// tiles of 64 along the long side that a CTA of a cluster of c can hold, with the short side of b
// tiles: beside X (hi and lo) lie S, the sums that the cluster exchanges and (b = 1) those that halves of a CTA do
int most_tiles(int b, int c) {
    const int s = 2 * b * b, exchange = c > 1 ? 2 * b * b : 0, halves = b == 1 ? 4 : 0;
    return ((int)kTiles - s - exchange - halves) / (2 * b);
}

__device__ __forceinline__ uint32_t rank_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void put_in_cluster(uint32_t addr, uint4 v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
template <int kC>
__device__ __forceinline__ void all_sync() {
    __syncwarp();
    if constexpr (kC > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();
}
// generic writes to shared memory, of this CTA or of any of the cluster, before the tensor core reads them
__device__ __forceinline__ void fence_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.proxy.async.shared::cluster;" ::: "memory"); }

// descriptor low word of an MN-major operand whose 64-row parts of M lie `apart` bytes from one another
__device__ __forceinline__ uint32_t mn_desc(uint32_t addr, uint32_t apart) {
    return ((apart >> 4) << 16) | ((addr & 0x3FFFFu) >> 4);
}

// An operand of 64 contraction indices: descriptors of its parts, and what a slice of 16 advances them.
struct Op {
    uint32_t hi, lo, step;
};

// Up to 64 indices in slices of 16, by a whole warp: small terms (lo lo too: 2.0e-6 instead of 2.2e-6
// off for 256 x 64), then hi hi, into an accumulator of its own.
__device__ __forceinline__ void issue(uint32_t d, const Op& p, const Op& q, int slices, uint32_t idesc, uint32_t leader) {
    if (slices == 4) {
        uint32_t acc = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk, acc = 1u)
                mma<1>(d, (i == 1 || i == 3 ? p.hi : p.lo) + kk * p.step, (i >= 2 ? q.hi : q.lo) + kk * q.step, idesc, acc, leader);
        return;
    }
    uint32_t acc = 0u;
    for (int i = 0; i < 4; ++i)
        for (int kk = 0; kk < slices; ++kk, acc = 1u)
            mma<1>(d, (i == 1 || i == 3 ? p.hi : p.lo) + kk * p.step, (i >= 2 ? q.hi : q.lo) + kk * q.step, idesc, acc, leader);
}
// slices that indices [64 t, n) of a tile have
__device__ __forceinline__ int slices_of(int n, int t) { return min(4, (n - 64 * t + 15) / 16); }

// After a wait that ran out: the MMAs that are still in flight are waited for (bounded), so that none of them
// writes tensor memory that another kernel has by then.  bars: the accumulators' two, and one for this.
__device__ __forceinline__ void finish(uint64_t* bars, bool aborted, int warp, uint32_t leader, uint32_t* status) {
    if (!aborted || warp != 0) return;
    commit<1>(&bars[2], leader);
    if (leader != 0u) wait_drain(&bars[2], 0, status);
    __syncwarp();
}

// a warp's sum, in all its lanes
__device__ __forceinline__ Sum warp_total(Sum s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float l = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
        s.add(__shfl_xor_sync(0xFFFFFFFFu, s.hi, o));
        s.lo += l;
    }
    if (__any_sync(0xFFFFFFFFu, s.wide != 0.0))         // NaN too
        for (int o = 16; o > 0; o >>= 1) s.wide += __shfl_xor_sync(0xFFFFFFFFu, s.wide, o);
    return s;
}

// U of this CTA's tiles, its norm over the cluster, and their images.  place(tile, row, col, at): the
// tile's first row and column, and where it lies behind x_hi (its low part x_lo bytes further).
template <int kC, typename A, typename F>
__device__ __forceinline__ void load_slab(const A& a, const Shape& shape, const Source& src, int b, int tiles,
                                          Partial* sums, float2* found, F place, uint8_t* x_hi, uint32_t x_lo) {
    const int groups = tiles * 512;             // of eight columns
    auto locate = [&](int g, int& row, int& col, uint32_t& at) {
        const int r = (g >> 3) & 63, q = g & 7;
        place(g >> 9, row, col, at);
        row += r;
        col += 8 * q;
        at += piece(r, q);
    };
    // kAhead groups of a thread at a time; where that is all, U stays in registers
    constexpr int kAhead = 4;
    float u[kAhead][8], kept[kAhead][8];
    auto read = [&](int g0) {
        Raws<kAhead> raw;
        raw.get(src, b, shape.cols, [&](int i, int& row, int& col) {
            uint32_t at;
            const int g = g0 + i * kThreads;
            if (g < groups) locate(g, row, col, at);
            return g < groups && row < shape.rows && col < shape.cols;
        });
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw.update(a.mu, a.nesterov, src, i, u[i], kept[i]);
    };
    Sum sum;
    for (int g0 = threadIdx.x; g0 < groups; g0 += kAhead * kThreads) {
        read(g0);
#pragma unroll
        for (int i = 0; i < kAhead; i += 2) sum.squares16(u[i]);
    }
    __shared__ Partial of_warp[kWarps];
    const int lane = threadIdx.x & 31;
    sum = warp_total(sum);
    if (lane == 0) of_warp[threadIdx.x >> 5] = Partial{sum.hi, sum.lo, sum.wide};
    __syncthreads();
    Sum total;
    if (threadIdx.x < 32) {
        if (lane < kWarps) {
            total.hi = of_warp[lane].hi;
            total.lo = of_warp[lane].lo;
            total.wide = of_warp[lane].wide;
        }
        total = warp_total(total);
    }
    if constexpr (kC > 1) {
        if (threadIdx.x < kC) {
            const Partial mine{total.hi, total.lo, total.wide};
            uint4 bits;
            memcpy(&bits, &mine, sizeof(bits));
            put_in_cluster(in_cta(smem_u32(&sums[rank_in_cluster()]), threadIdx.x), bits);
        }
        all_sync<kC>();
        total = Sum();
        if (threadIdx.x == 0)
            for (int c = 0; c < kC; ++c) {
                total.add(sums[c].hi);
                total.lo += sums[c].lo;
                total.wide += sums[c].wide;
            }
    }
    if (threadIdx.x == 0) *found = factors(total, a.eps);
    __syncthreads();
    const float2 factor = *found;
    for (int g0 = threadIdx.x; g0 < groups; g0 += kAhead * kThreads) {
        if (groups > kAhead * kThreads) read(g0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int g = g0 + i * kThreads;
            if (g >= groups) continue;
            int row, col;
            uint32_t at;
            locate(g, row, col, at);
            const bool inside = row < shape.rows && col < shape.cols;
            if (inside && src.m.data != nullptr) put8(src.out, b, row, col, shape.cols, kept[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i][e] = inside && col + e < shape.cols ? u[i][e] * factor.x * factor.y : 0.f;
            uint4 hi, lo;
            split8(u[i], hi, lo);
            *reinterpret_cast<uint4*>(x_hi + at) = hi;
            *reinterpret_cast<uint4*>(x_hi + x_lo + at) = lo;
        }
    }
    fence_shared();
    __syncthreads();
}

// The short side 65 to 128: kB tiles of 64.  kC: CTAs a cluster
template <int kC>
__global__ void __launch_bounds__(kThreads, 1) small_kernel(const __grid_constant__ SmallArgs a) {
    constexpr int kB = 2;
    constexpr int kM = 64 * kB;                 // rows of S
    constexpr int kCols = 16 * kB;              // of a thread, in S
    constexpr int kOwn = kM / kC;               // rows of S that a CTA adds up
    constexpr int kAtOnce = 2;                  // tiles of the long side at once in P X
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem);                   // [3] of the accumulators' two buffers, and to drain
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + 24);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + 28);
    float2* const found = reinterpret_cast<float2*>(smem + 32);
    Partial* const sums = reinterpret_cast<Partial*>(smem + 64);                // [kC]
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = kC > 1 ? rank_in_cluster() : 0u;

    if (threadIdx.x == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        mbar_init(&bars[2], 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(2 * kHalfTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    all_sync<kC>();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();

    // this cluster's matrix and this CTA's slab
    const uint32_t matrix = blockIdx.x / kC;
    const int k = element_of(a.n, matrix, [&](int i) { return a.shape[i].first[0]; });
    const Shape shape = a.shape[k];
    const Source src = a.source[k];
    const int b = (int)(matrix - shape.first[0]);
    const bool wide = shape.rows <= shape.cols;
    const int m = min(shape.rows, shape.cols), tiles = tiles_of(max(shape.rows, shape.cols));
    const int nt_most = (tiles + kC - 1) / kC;
    const int t0 = tiles * (int)rank / kC, nt = tiles * ((int)rank + 1) / kC - t0;
    // tile (along the short side s, along the long one t): rows of K-major operands follow one another
    const uint32_t t_step = (wide ? kB : 1) * kTileBytes, s_step = (wide ? 1 : nt_most) * kTileBytes;
    uint8_t* const x_hi = smem + kHeader;
    uint8_t* const s_hi = x_hi + (size_t)2 * nt_most * kB * kTileBytes;
    uint8_t* const exchange = s_hi + 2 * kB * kB * kTileBytes;
    const uint32_t x_lo = (uint32_t)(nt_most * kB) * kTileBytes, s_lo = kB * kB * kTileBytes;    // from hi to lo
    const uint32_t xa = smem_u32(x_hi), sa = smem_u32(s_hi);
    auto tile_at = [&](int s, int t) { return (uint32_t)s * s_step + (uint32_t)t * t_step; };

    load_slab<kC>(a, shape, src, b, nt * kB, sums, found,
                      [&](int tile, int& row, int& col, uint32_t& at) {
                          const int sh = tile % kB, t = tile / kB;
                          row = (wide ? sh : t0 + t) * 64;
                          col = (wide ? t0 + t : sh) * 64;
                          at = tile_at(sh, t);
                      },
                      x_hi, x_lo);

    // ---- the steps
    const uint32_t leader = lane == 0 ? 1u : 0u;
    const int quad = warp & 3, part_of = warp >> 2, r = 32 * quad + lane;  // row of the accumulators, quarter of their columns
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    uint32_t parity = 0;                        // a bit for each buffer
    auto wait = [&](int z) {
        wait_bounded(&bars[z], (parity >> z) & 1u, abort_flag, a.status, kStatusTimeoutMma);
        parity ^= 1u << z;
        tc_fence_after();
    };
    constexpr uint32_t kF32 = 1u << 4, kM128 = (uint32_t)(128 >> 4) << 24;
    const uint32_t square_desc = kF32 | kM128 | ((uint32_t)(kM >> 3) << 17);
    const uint32_t gram_desc = square_desc | (wide ? 0u : (1u << 15) | (1u << 16));
    // S's rows by 64 columns from column tile t on
    auto sym = [&](int t) {
        const uint32_t at = sa + (uint32_t)(t * kB) * kTileBytes;
        return Op{sdesc128_lo(at), sdesc128_lo(at + s_lo), 2u};
    };
    // a thread's columns of S from accumulators, added to v or put there
    auto drain = [&](uint32_t from, float* v, bool add) {
        uint32_t bits[kCols];
        tmem_ld32(from, bits);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < kCols; ++e) v[e] = add ? v[e] + __uint_as_float(bits[e]) : __uint_as_float(bits[e]);
    };
    // what sums over the long and the short side are short of (see uncut())
    const int n_slices = slices_of(max(shape.rows, shape.cols), 0), m_slices = slices_of(m, 0);
    const float n_short = short_of(n_slices), m_short = short_of(m_slices);
    const int col0 = part_of * kCols;           // of S

    for (int step = 0; step < a.steps; ++step) {
        const float ca = a.abc[3 * step], cb = a.abc[3 * step + 1], cc = a.abc[3 * step + 2];
        // S: this slab's part, a tile of the long side at a time
        float part[kCols];
#pragma unroll
        for (int e = 0; e < kCols; ++e) part[e] = 0.f;
        auto gram = [&](int t) {
            const uint32_t at = xa + (uint32_t)t * t_step;
            Op o;
            if (wide) o = Op{sdesc128_lo(at), sdesc128_lo(at + x_lo), 2u};
            else o = Op{mn_desc(at, s_step), mn_desc(at + x_lo, s_step), 128u};
            issue(tmem + (uint32_t)(t & 1) * kHalfTmem, o, o, slices_of(max(shape.rows, shape.cols), t0 + t), gram_desc, leader);
            commit<1>(&bars[t & 1], leader);
        };
        if (warp == 0) {
            tc_fence_after();
            for (int t = 0; t < min(nt, 2); ++t) gram(t);
        }
        for (int t = 0; t < nt; ++t) {
            wait(t & 1);
            drain(lanes + (uint32_t)(t & 1) * kHalfTmem + (uint32_t)col0, part, true);
            tc_fence_before();
            __syncthreads();
            if (warp == 0 && t + 2 < nt) {
                tc_fence_after();
                gram(t + 2);
            }
        }
        if constexpr (kC > 1) {
            // to the CTA that adds up the row
            const uint32_t to = in_cta(smem_u32(exchange), (uint32_t)(r / kOwn)) +
                                (uint32_t)(((int)rank * kOwn + r % kOwn) * kM + col0) * 4u;
#pragma unroll
            for (int c = 0; c < kCols; c += 4)
                put_in_cluster(to + 4u * c, make_uint4(__float_as_uint(part[c]), __float_as_uint(part[c + 1]),
                                                       __float_as_uint(part[c + 2]), __float_as_uint(part[c + 3])));
            all_sync<kC>();
            for (int v = threadIdx.x; v < kOwn * kM / 8; v += kThreads) {
                const int own = v / (kM / 8), col = v % (kM / 8) * 8, row = (int)rank * kOwn + own;
                float s[8];
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const float4* f = reinterpret_cast<const float4*>(exchange) + ((c * kOwn + own) * kM + col) / 4;
                    const float4 x = f[0], y = f[1];
                    const float p[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = c == 0 ? p[e] : s[e] + p[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = uncut(s[e], n_short) * kUnscale;
                uint4 hi, lo;
                split8(s, hi, lo);
                const uint32_t at = sa + (uint32_t)(col / 64 * kB + row / 64) * kTileBytes + piece(row & 63, (col & 63) >> 3);
#pragma unroll
                for (uint32_t c = 0; c < kC; ++c) {
                    const uint32_t to = in_cta(at, c);
                    put_in_cluster(to, hi);
                    put_in_cluster(to + s_lo, lo);
                }
            }
            fence_cluster();
            all_sync<kC>();
            fence_cluster();
        } else {
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
                const int col = col0 + c;
#pragma unroll
                for (int e = 0; e < 8; ++e) part[c + e] = uncut(part[c + e], n_short) * kUnscale;
                uint4 hi, lo;
                split8(part + c, hi, lo);
                uint8_t* at = s_hi + (col / 64 * kB + r / 64) * kTileBytes + piece(r & 63, (col & 63) >> 3);
                *reinterpret_cast<uint4*>(at) = hi;
                *reinterpret_cast<uint4*>(at + s_lo) = lo;
            }
            fence_shared();
            __syncthreads();
        }

        // P = a I + b S + c S S, over S
        if (warp == 0) {
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < kB; ++t) issue(tmem + (uint32_t)t * kHalfTmem, sym(t), sym(t), slices_of(m, t), square_desc, leader);
            commit<1>(&bars[0], leader);
        }
        wait(0);
        drain(lanes + (uint32_t)col0, part, false);
        drain(lanes + kHalfTmem + (uint32_t)col0, part, true);
        tc_fence_before();
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
            const int col = col0 + c;
            uint8_t* at = s_hi + (col / 64 * kB + r / 64) * kTileBytes + piece(r & 63, (col & 63) >> 3);
            float s[8];
            join8(*reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + s_lo), s);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] = fmaf(cc, uncut(part[c + e], m_short) * kUnscale, cb * s[e]);
                if (r == col + e && r < m) s[e] += ca * kScale;
            }
            uint4 hi, lo;
            split8(s, hi, lo);
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + s_lo) = lo;
        }
        fence_shared();
        __syncthreads();

        // P X over X, some tiles of the long side at a time: 64 x 64 blocks of the result, each
        // from kB slices of 64 indices in accumulators of their own
        const bool last = step == a.steps - 1;
        const int passes = (nt + kAtOnce - 1) / kAtOnce;
        auto update = [&](int n) {
            const uint32_t d = tmem + (uint32_t)(n & 1) * kHalfTmem;
            const int first = n * kAtOnce, count = min(kAtOnce, nt - first);
            for (int s = 0; s < kB; ++s) {
                if (wide) {
                    const uint32_t at = xa + tile_at(s, first);
                    const Op q{mn_desc(at, t_step), mn_desc(at + x_lo, t_step), 128u};
                    issue(d + (uint32_t)s * 128u, sym(s), q, slices_of(m, s), kF32 | kM128 | (1u << 16) | ((uint32_t)(8 * count) << 17), leader);
                } else {
                    const uint32_t at = xa + tile_at(s, first);
                    const Op p{sdesc128_lo(at), sdesc128_lo(at + x_lo), 2u};
                    issue(d + (uint32_t)s * 128u, p, sym(s), slices_of(m, s), square_desc, leader);
                }
            }
            commit<1>(&bars[n & 1], leader);
        };
        if (warp == 0) {
            tc_fence_after();
            for (int n = 0; n < min(passes, 2); ++n) update(n);
        }
        for (int n = 0; n < passes; ++n) {
            wait(n & 1);
            const int first = n * kAtOnce;
            // a thread's columns of its row: a quarter of the accumulators', in one tile
            constexpr int kWidth = 64 / kB;
            const int block = part_of / kB, c0 = part_of % kB * kWidth;     // of 64 columns; first one in it
            const uint32_t from = lanes + (uint32_t)(n & 1) * kHalfTmem + (uint32_t)(block * 64 + c0);
            float f[kWidth];
            {
                uint32_t bits[64];
                tmem_ld32(from, bits);
                tmem_ld32(from + 128u, bits + 32);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < kWidth; ++e) f[e] = uncut(__uint_as_float(bits[e]) + __uint_as_float(bits[32 + e]), m_short);
            }
            const int s = wide ? r / 64 : block, t = first + (wide ? block : r / 64);
            if (t < nt) {                                   // (the same for a warp)
                uint8_t* const tile = x_hi + tile_at(s, t);
                if (last) {
                    // by way of what these 32 rows of X were (hi or lo part, as two warps have a tile's
                    // rows): nobody reads them any more
                    const Result& o = a.result[k];
                    uint8_t* const stage = tile + 4096 * (quad & 1) + (c0 != 0 ? x_lo : 0u);
                    const int row0 = (wide ? s : t0 + t) * 64 + 32 * (quad & 1), first_col = (wide ? t0 + t : s) * 64 + c0;
                    if (first_col < shape.cols) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float* v = f + 4 * q;
                            const float by = kUnscale * kUnscale;
                            *reinterpret_cast<float4*>(stage + staged<32>(lane, q)) =
                                make_float4(o.beta * (v[0] * by), o.beta * (v[1] * by), o.beta * (v[2] * by), o.beta * (v[3] * by));
                        }
                        __syncwarp();
                        write_rows<32, 1>(a.alpha, o, b, row0, first_col, shape.rows, shape.cols, stage, lane);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < kWidth / 8; ++q) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[8 * q + e] *= kUnscale;
                        uint4 hi, lo;
                        split8(f + 8 * q, hi, lo);
                        uint8_t* at = tile + piece(r & 63, c0 / 8 + q);
                        *reinterpret_cast<uint4*>(at) = hi;
                        *reinterpret_cast<uint4*>(at + x_lo) = lo;
                    }
                }
            }
            tc_fence_before();
            if (n == passes - 1) fence_shared();
            __syncthreads();
            if (warp == 0 && n + 2 < passes) {
                tc_fence_after();
                update(n + 2);
            }
        }
    }

    finish(bars, *abort_flag != 0, warp, leader, a.status);
    all_sync<kC>();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kHalfTmem));
    }
}

// The short side at most 64.  A tile's hi and lo lie behind one another and are one operand of 128
// rows: one MMA gives hi hi, hi lo, lo hi and lo lo in the quarters of its accumulators (rows 0-63
// and 64-127, columns 0-63 and 64-127), which are added up outside: a quarter of the MMAs, and the
// small terms by themselves.  Warps of rows r and 64 + r change halves of what they have: a thread
// ends up with 8 elements of one row, a piece of an image.  (A warp of its own for the MMAs leaves
// 96 registers a thread, whose spills cost more than it gives.)
template <int kC>
__global__ void __launch_bounds__(kThreads, 1) narrow_kernel(const __grid_constant__ SmallArgs a) {
    constexpr uint32_t kPair = 2 * kTileBytes;
    constexpr int kOwn = 64 / kC;               // rows of S that a CTA adds up
    constexpr int kAtOnce = 2;                  // tiles of P X at once, in each of two buffers
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem);                   // [3] of the accumulators' two buffers, and to drain
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + 24);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + 28);
    float2* const found = reinterpret_cast<float2*>(smem + 32);
    Partial* const sums = reinterpret_cast<Partial*>(smem + 64);                // [kC]
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = kC > 1 ? rank_in_cluster() : 0u;

    if (threadIdx.x == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        mbar_init(&bars[2], 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(2 * kHalfTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    all_sync<kC>();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();

    const uint32_t matrix = blockIdx.x / kC;
    const int k = element_of(a.n, matrix, [&](int i) { return a.shape[i].first[0]; });
    const Shape shape = a.shape[k];
    const Source src = a.source[k];
    const int b = (int)(matrix - shape.first[0]);
    const bool wide = shape.rows <= shape.cols;
    const int m = min(shape.rows, shape.cols), n = max(shape.rows, shape.cols), tiles = tiles_of(n);
    const int nt_most = (tiles + kC - 1) / kC;
    const int t0 = tiles * (int)rank / kC, nt = tiles * ((int)rank + 1) / kC - t0;
    uint8_t* const x = smem + kHeader;          // pairs of tiles along the long side
    uint8_t* const sp = x + (size_t)nt_most * kPair;
    float4* const halves = reinterpret_cast<float4*>(sp + kPair);               // [4][kThreads]
    uint8_t* const exchange = sp + 3 * kPair;
    const uint32_t xa = smem_u32(x), sa = smem_u32(sp);

    load_slab<kC>(a, shape, src, b, nt, sums, found,
                  [&](int t, int& row, int& col, uint32_t& at) {
                      row = wide ? 0 : (t0 + t) * 64;
                      col = wide ? (t0 + t) * 64 : 0;
                      at = (uint32_t)t * kPair;
                  },
                  x, kTileBytes);

    const uint32_t leader = lane == 0 ? 1u : 0u;
    const int quad = warp & 3, part = warp >> 2, low = quad >> 1;
    const int r = 32 * (quad & 1) + lane;       // this thread's row
    const int q = 2 * part + low;               // and piece of it: columns 8 q to 8 q + 7
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t own_piece = piece(r, q);
    uint32_t parity = 0;                        // a bit for each buffer
    auto wait = [&](int z) {
        wait_bounded(&bars[z], (parity >> z) & 1u, abort_flag, a.status, kStatusTimeoutMma);
        parity ^= 1u << z;
        tc_fence_after();
    };
    // the four quarters' terms of this thread's 8 elements (v), of kT tiles whose accumulators lie
    // 128 columns apart, or (added) of the sum over two accumulators, or four
    auto gather = [&](uint32_t from, auto tiles_of_it, int added, float* v) {
        constexpr int kT = decltype(tiles_of_it)::value;
        float all[kT][16];
        {
            uint32_t lead[kT][16], rest[kT][16];
#pragma unroll
            for (int i = 0; i < kT; ++i) {
                tmem_ld16(from + (uint32_t)(128 * i + 16 * part), lead[i]);
                tmem_ld16(from + (uint32_t)(128 * i + 64 + 16 * part), rest[i]);
            }
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) all[i][e] = __uint_as_float(lead[i][e]) + __uint_as_float(rest[i][e]);
        }
        const bool both = kT == 2 && added > 0;
        if (both) {
#pragma unroll
            for (int e = 0; e < 16; ++e) all[0][e] += all[kT - 1][e];
#pragma unroll 1
            for (int i = kT; i < added; ++i) {
                uint32_t lead[16], rest[16];
                tmem_ld16(from + (uint32_t)(128 * i + 16 * part), lead);
                tmem_ld16(from + (uint32_t)(128 * i + 64 + 16 * part), rest);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) all[0][e] += __uint_as_float(lead[e]) + __uint_as_float(rest[e]);
            }
        }
        // rows r give away columns 8-15 of the 16 they have, rows 64 + r columns 0-7
#pragma unroll
        for (int i = 0; i < kT; ++i) {
            if (i > 0 && both) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* lower = all[i] + 4 * h;
                halves[(2 * i + h) * kThreads + threadIdx.x] =
                    make_float4(low ? lower[0] : lower[8], low ? lower[1] : lower[9], low ? lower[2] : lower[10], low ? lower[3] : lower[11]);
            }
        }
        asm volatile("bar.sync %0, 64;" ::"r"(1 + 2 * part + (quad & 1)) : "memory");
#pragma unroll
        for (int i = 0; i < kT; ++i) {
            if (i > 0 && both) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 f = halves[(2 * i + h) * kThreads + (threadIdx.x ^ 64)];
                const float g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) v[8 * i + 4 * h + e] = g[e] + (low ? all[i][8 + 4 * h + e] : all[i][4 * h + e]);
            }
        }
        // (the exchange may be written again behind the next barrier of the CTA only)
    };
    constexpr std::integral_constant<int, 1> kOne{};
    constexpr std::integral_constant<int, 2> kTwo{};
    auto put8_pair = [&](uint8_t* pair, const float* v) {
        uint4 hi, lo;
        split8(v, hi, lo);
        *reinterpret_cast<uint4*>(pair + own_piece) = hi;
        *reinterpret_cast<uint4*>(pair + kTileBytes + own_piece) = lo;
    };
    constexpr uint32_t kDesc = (1u << 4) | ((uint32_t)(128 >> 4) << 24);        // fp32 accumulators, M = 128
    constexpr uint32_t kN128 = (uint32_t)(128 >> 3) << 17, kAMn = 1u << 15, kBMn = 1u << 16;
    // products of pairs, in slices of 16 indices
    auto multiply = [&](uint32_t d, uint32_t p, uint32_t p_step, uint32_t q0, uint32_t q_step, int slices, uint32_t idesc,
                        uint32_t acc) {
        if (slices == 4) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk, acc = 1u) mma<1>(d, p + kk * p_step, q0 + kk * q_step, idesc, acc, leader);
            return;
        }
        for (int kk = 0; kk < slices; ++kk, acc = 1u) mma<1>(d, p + kk * p_step, q0 + kk * q_step, idesc, acc, leader);
    };
    const int m_slices = slices_of(m, 0);
    const float m_short = short_of(m_slices);
    // accumulators of S, of two tiles each or few more: a sum is cut off at every addition (9 x 423 with four
    // tiles in one: 1.5 times as far off as fp32 products, so 1.2); additions into one
    const int apart = nt_most <= 4 ? 2 : 4;
    const float n_short = nt_most > 1 ? short_of(4 * ((nt_most + apart - 1) / apart)) : short_of(slices_of(n, 0));

    for (int step = 0; step < a.steps; ++step) {
        const float ca = a.abc[3 * step], cb = a.abc[3 * step + 1], cc = a.abc[3 * step + 2];
        // S: this slab's part, its tiles in turn into the accumulators
        if (warp == 0) {
            tc_fence_after();
            for (int t = 0; t < nt; ++t) {
                const uint32_t at = xa + (uint32_t)t * kPair;
                const uint32_t o = wide ? sdesc128_lo(at) : sdesc128mn_lo(at);
                multiply(tmem + (uint32_t)(t & (apart - 1)) * 128u, o, wide ? 2u : 128u, o, wide ? 2u : 128u, slices_of(n, t0 + t),
                         kDesc | kN128 | (wide ? 0u : kAMn | kBMn), t < apart ? 0u : 1u);
            }
            commit<1>(&bars[0], leader);
        }
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.f;
        wait(0);
        if (nt > 1) {
            float v[16];
            gather(lanes, kTwo, min(apart, nt), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = v[e];
        } else if (nt == 1) {
            gather(lanes, kOne, 0, s);
        }
        tc_fence_before();
        if constexpr (kC > 1) {
            // to the CTA that adds up the row
            const uint32_t to = in_cta(smem_u32(exchange), (uint32_t)(r / kOwn)) + (uint32_t)(((int)rank * kOwn + r % kOwn) * 64 + 8 * q) * 4u;
            put_in_cluster(to, make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]), __float_as_uint(s[3])));
            put_in_cluster(to + 16u, make_uint4(__float_as_uint(s[4]), __float_as_uint(s[5]), __float_as_uint(s[6]), __float_as_uint(s[7])));
            all_sync<kC>();
            if ((int)threadIdx.x < kOwn * 8) {
                const int own = threadIdx.x >> 3, piece_of = threadIdx.x & 7, row = (int)rank * kOwn + own;
                float f[8];
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const float4* from = reinterpret_cast<const float4*>(exchange) + ((c * kOwn + own) * 64 + 8 * piece_of) / 4;
                    const float4 y = from[0], z = from[1];
                    const float g[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = c == 0 ? g[e] : f[e] + g[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = uncut(f[e], n_short) * kUnscale;
                uint4 hi, lo;
                split8(f, hi, lo);
#pragma unroll
                for (uint32_t c = 0; c < kC; ++c) {
                    const uint32_t to_s = in_cta(sa + piece(row, piece_of), c);
                    put_in_cluster(to_s, hi);
                    put_in_cluster(to_s + kTileBytes, lo);
                }
            }
            fence_cluster();
            all_sync<kC>();
            fence_cluster();
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = uncut(s[e], n_short) * kUnscale;
            put8_pair(sp, s);
            fence_shared();
            __syncthreads();
        }

        // P = a I + b S + c S S, over S
        const uint32_t sd = sdesc128_lo(sa);
        if (warp == 0) {
            tc_fence_after();
            multiply(tmem, sd, 2u, sd, 2u, m_slices, kDesc | kN128, 0u);
            commit<1>(&bars[0], leader);
        }
        wait(0);
        float p[8];
        gather(lanes, kOne, 0, p);
        tc_fence_before();
        join8(*reinterpret_cast<const uint4*>(sp + own_piece), *reinterpret_cast<const uint4*>(sp + kTileBytes + own_piece), s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = fmaf(cc, uncut(p[e], m_short) * kUnscale, cb * s[e]);
            if (r == 8 * q + e && r < m) p[e] += ca * kScale;
        }
        put8_pair(sp, p);
        fence_shared();
        __syncthreads();

        // P X over X
        const bool last = step == a.steps - 1;
        const int passes = (nt + kAtOnce - 1) / kAtOnce;
        auto update = [&](int pass) {
            for (int i = 0; i < kAtOnce && pass * kAtOnce + i < nt; ++i) {
                const uint32_t at = xa + (uint32_t)(pass * kAtOnce + i) * kPair;
                const uint32_t d = tmem + (uint32_t)(pass & 1) * kHalfTmem + 128u * i;
                if (wide) multiply(d, sd, 2u, sdesc128mn_lo(at), 128u, m_slices, kDesc | kN128 | kBMn, 0u);
                else multiply(d, sdesc128_lo(at), 2u, sd, 2u, m_slices, kDesc | kN128, 0u);
            }
            commit<1>(&bars[pass & 1], leader);
        };
        if (warp == 0) {
            tc_fence_after();
            for (int pass = 0; pass < min(passes, 2); ++pass) update(pass);
        }
        for (int pass = 0; pass < passes; ++pass) {
            wait(pass & 1);
            const int first = pass * kAtOnce, count = min(kAtOnce, nt - first);
            const uint32_t from = lanes + (uint32_t)(pass & 1) * kHalfTmem;
            float v[16];
            if (count == 2) gather(from, kTwo, 0, v);
            else gather(from, kOne, 0, v);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (i >= count) break;
                uint8_t* const pair = x + (size_t)(first + i) * kPair;
                float* f = v + 8 * i;
                if (!last) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = uncut(f[e], m_short) * kUnscale;
                    put8_pair(pair, f);
                } else {
                    // fp32 in the place of the pair, as two blocks of 32 columns
                    const float by = a.result[k].beta;
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = by * (uncut(f[e], m_short) * (kUnscale * kUnscale));
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float4*>(pair + (q >> 2) * kTileBytes + staged<32>(r, 2 * (q & 3) + h)) =
                            make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
                }
            }
            tc_fence_before();
            if (pass == passes - 1) fence_shared();
            __syncthreads();
            if (warp == 0 && pass + 2 < passes) {
                tc_fence_after();
                update(pass + 2);
            }
            if (last && warp < 4 * count) {
                // a warp for 32 rows of 32 columns
                const Result& o = a.result[k];
                const int i = warp >> 2, rows = warp & 1, cols = (warp >> 1) & 1;
                const int row0 = (wide ? 0 : (t0 + first + i) * 64) + 32 * rows, col0 = (wide ? (t0 + first + i) * 64 : 0) + 32 * cols;
                if (col0 < shape.cols && row0 < shape.rows)
                    write_rows<32, 1>(a.alpha, o, b, row0, col0, shape.rows, shape.cols,
                                   x + (size_t)(first + i) * kPair + cols * kTileBytes + 4096 * rows, lane);
            }
        }
    }

    finish(bars, *abort_flag != 0, warp, leader, a.status);
    all_sync<kC>();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kHalfTmem));
    }
}

// ---------------------------------------------------------------- host

template <int kC, int kB>
cudaError_t run(unsigned matrices, cudaStream_t s, const SmallArgs& args) {
    void (*kernel)(SmallArgs) = nullptr;
    if constexpr (kB == 1) kernel = narrow_kernel<kC>;
    else kernel = small_kernel<kC>;
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !allowed[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[dev] = true;
    }
    return launch_clusters(kernel, matrices * kC, kThreads, kSmem, kC, s, args);
}

template <int kB>
cudaError_t run(int c, unsigned matrices, cudaStream_t s, const SmallArgs& args) {
    switch (c) {
        case 1: return run<1, kB>(matrices, s, args);
        case 2: return run<2, kB>(matrices, s, args);
        case 4: return run<4, kB>(matrices, s, args);
        default: return run<8, kB>(matrices, s, args);
    }
}

int short_tiles(const mttkrp_matrices& m) { return tiles_of((int)std::min(m.rows, m.cols)); }
int long_tiles(const mttkrp_matrices& m) { return tiles_of((int)std::max(m.rows, m.cols)); }

// CTAs for a matrix: one where it does with few tiles (an exchange over a cluster is as long as
// the work on four or eight), else as many as leave each two or four while there are SMs for all, and
// as hold it in any case.
int cluster_of(const mttkrp_matrices& m, int64_t matrices, int sms) {
    const int b = short_tiles(m), t = long_tiles(m), alone = b == 1 ? 8 : 3, each = b == 1 ? 4 : 2;
    int c = 1;
    while (c < 8 && most_tiles(b, c) * c < t) c *= 2;
    while (c < 8 && t > alone && t > each * c && matrices * c * 2 <= sms) c *= 2;
    return c;
}

cudaError_t run_list(const NewtonArgs& a, int64_t matrices, int sms, cudaStream_t s) {
    SmallArgs p;
    p.steps = a.steps;
    p.mu = a.mu;
    p.alpha = a.alpha;
    p.nesterov = a.nesterov;
    p.eps = a.eps;
    p.status = a.status;
    for (int i = 0; i < 3 * a.steps; ++i) p.abc[i] = a.coefficients[i];
    cudaError_t e = cudaSuccess;
    // a launch for every size of cluster and short side, of as many elements as a table holds and as many
    // matrices as a grid
    for (int b = 1; b <= 2; ++b)
        for (int c = 1; c <= 8; c *= 2)
            deal(
                a.n, kElements, INT32_MAX / c,
                [&](int k) {
                    const mttkrp_matrices& m = a.grad[k];
                    const bool here = newton_some(m) && newton_is_small(m) && short_tiles(m) == b && cluster_of(m, matrices, sms) == c;
                    return here ? m.batch : 0;
                },
                [&](int i, int k, int64_t b0, int64_t count, int64_t before) {
                    const mttkrp_matrices& m = a.grad[k];
                    p.shape[i] = Shape{0, (int)m.rows, (int)m.cols, (int)count, {(uint32_t)before, 0}};
                    Source& u = p.source[i];
                    u.g = store_of(m, b0);
                    u.m = u.out = Store{nullptr, 0, 0, 0, 0};
                    if (a.momentum != nullptr) {
                        u.m = store_of(a.momentum[k], b0);
                        u.out = store_of(a.momentum_out[k], b0);
                    }
                    Result& r = p.result[i];
                    r.out = store_of(a.out[k], b0);
                    r.w = a.weight != nullptr ? store_of(a.weight[k], b0) : Store{nullptr, 0, 0, 0, 0};
                    r.beta = a.beta[k];
                },
                [&](int parts, int64_t used) {
                    p.n = parts;
                    if (e == cudaSuccess) e = b == 1 ? run<1>(c, (unsigned)used, s, p) : run<2>(c, (unsigned)used, s, p);
                    return e == cudaSuccess;
                });
    return e;
}

}  // namespace

bool newton_is_small(const mttkrp_matrices& m) {
    const int b = short_tiles(m);
    return b <= 2 && long_tiles(m) <= 8 * most_tiles(b, 8);
}

cudaError_t launch_newton_small(const NewtonArgs& a, int sms, cudaStream_t s) {
    int64_t matrices = 0;
    for (int k = 0; k < a.n; ++k)
        if (newton_some(a.grad[k]) && newton_is_small(a.grad[k])) matrices += a.grad[k].batch;
    return matrices > 0 ? run_list(a, matrices, sms, s) : cudaSuccess;
}

}  // namespace mk
