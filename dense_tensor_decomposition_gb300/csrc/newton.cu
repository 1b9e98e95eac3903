// Orthogonalisation by Newton-Schulz products: X = U / (|U|_F + eps), then every step
//   S = X X^T (of the smaller side, m),  P = a I + b S + c S S,  X <- P X
// (for more rows than columns S = X^T X and X <- X P).
//
// Arithmetic.  The products run on the tensor cores in fp16 with fp32 accumulation, on
// operands split in two: x 2^12 = hi + lo, 22 bits in all.  hi hi + hi lo + lo hi is then an
// fp32 product to about 2^-22; sums in tensor memory are cut off towards zero at every
// addition, so that they go to fp32 registers every 128 indices.  That is what results in fp32
// and fp16 get.  For results in bf16 two terms less do: S and S S from hi hi alone, P X from
// P's hi with both parts of X.  What must keep its low part is X: rounded to 11 bits, a
// gradient of few strong directions loses its weak ones, which the steps raise by up to 485
// times (relative errors at 512 x 512, 16 strong directions over noise of 1e-2: 2.4e-2 with
// everything from hi; 1e-3 so; rounding the result to bf16 is 1.7e-3 by itself).  And what S S
// loses with S's low part lies mostly on S's diagonal, far larger than the rest: the epilogue
// adds (lo_ii + lo_jj) hi_ij (256 x 1024, noise alone: 2.7e-3 without, 1.3e-3 with).  Singular
// values stay below 3.9 (checked on the host), so that nothing leaves fp16's range.
//
// Layout.  X, S and P live in the workspace as images: 64 x 64 tiles of 8 KB, hi and lo apart,
// rows of 128 bytes with their 16-byte pieces already in the order of the 128-byte swizzle.  A
// tile as it is serves as operand with K along its rows (K-major) or down its columns
// (MN-major), so nothing is transposed in memory, tall matrices need no other kernel than wide
// ones, and one tensor map over the workspace, as rows of 128 bytes, loads everything.  Of the
// symmetric S and P only blocks on and above the diagonal are computed and stored; a block
// below it is read as the MN-major form of its mirror image.
//
// A launch does one product for all matrices of a list: a CTA (or a pair of CTAs that share one
// tcgen05.mma, cta_group::2) takes tiles of the result in turn; a TMA thread fills a ring of
// stages of 64 contraction indices, one thread issues MMAs into one of two accumulators in tensor
// memory, eight or 16 warps drain the other one and write the result.  Which of the two forms
// runs is the host's choice, product by product (number_items, newton_plan.h).
//
// What bounds it, and measured (five steps, fp32 / bf16).  Large matrices: the tensor cores; 2 x
// 4096 x 4096 in 5.4 / 2.6 ms, 1520 TFLOP/s of MMAs done in fp32 (three an fp32 product), 80 % of a
// large library product's rate.  Tiles that do not fill the SMs a whole number of times:
// 12 x 1024 x 4096 2.2 / 1.15 ms, 8 x 2048 x 1360 1.67 / 0.85 ms.  Few tiles: launches of 11 to 17 us of
// which half is filling and draining; 3 x 512 x 2000 227 / 167 us.  Many small ones: epilogues and the
// passes over U; 64 x 501 x 333 485 / 339 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "launch.cuh"
#include "newton.cuh"
#include "newton.h"
#include "newton_plan.h"

namespace mk {
namespace {

constexpr int kMaxSlices = 256;             // CTAs a matrix in the passes over U
constexpr int64_t kGroupTiles = (int64_t)4 << 17;   // 4 GB of images a group (one matrix at least)

constexpr int kEpiWarp0 = 4;
constexpr int kPassThreads = 256;

// ---------------------------------------------------------------- the passes over U

// a sum of squares as fp32 pair, and in fp64 what does not fit
struct Partial {
    float hi, lo;
    double wide;
};

struct PassArgs {
    int n;
    float mu;
    bool nesterov;
    double eps;
    Partial* partial;
    uint8_t* tiles;
    Shape shape[kTable];
    Source source[kTable];
};

// Sums of squares: a matrix in slices of consecutive groups of 8 columns, row by row, a slice
// a CTA.
template <bool kMomentum>
__global__ void __launch_bounds__(kPassThreads) squares_kernel(const __grid_constant__ PassArgs a) {
    after_previous();
    const int k = element_of(a.n, blockIdx.x, [&](int i) { return a.source[i].first[0]; });
    const Source s = a.source[k];
    const int cols = a.shape[k].cols, per = (cols + 7) / 8;
    const uint32_t at = blockIdx.x - s.first[0];
    const int b = (int)(at / (uint32_t)s.slices), slice = (int)(at - (uint32_t)b * s.slices);
    const int64_t groups = (int64_t)a.shape[k].rows * per;
    const bool narrow = groups < INT32_MAX;
    const int64_t g0 = groups * slice / s.slices, g1 = groups * (slice + 1) / s.slices;
    Sum sum;
    constexpr int kAhead = kMomentum ? 2 : 4;
    for (int64_t g = g0 + threadIdx.x; g < g1; g += kAhead * kPassThreads) {
        Raws<kAhead, kMomentum> raw;
        raw.get(s, b, cols, [&](int i, int& r, int& c) {
            const int64_t x = g + i * kPassThreads;
            r = narrow ? (int)((uint32_t)x / (uint32_t)per) : (int)(x / per);
            c = (int)(x - (int64_t)r * per) * 8;
            return x < g1;
        });
#pragma unroll
        for (int i = 0; i < kAhead; i += 2) {
            float v[2][8], kept[8];
            raw.update(a.mu, a.nesterov, s, i, v[0], kept);
            raw.update(a.mu, a.nesterov, s, i + 1, v[1], kept);
            sum.squares16(v[0]);
        }
    }
    const Sum total = block_total<kPassThreads / 32>(sum);
    if (threadIdx.x == 0) a.partial[s.at + b * s.slices + slice] = Partial{total.hi, total.lo, total.wide};
}

// The images of X = U / (|U| + eps), zeros behind the last row and column; momentum written.
// A CTA takes 64 rows of four column tiles: a warp reads and writes one row of them at a time.
constexpr int kStrip = 4;

template <bool kMomentum>
__global__ void __launch_bounds__(kPassThreads) images_kernel(const __grid_constant__ PassArgs a) {
    after_previous();
    const int k = element_of(a.n, blockIdx.x, [&](int i) { return a.source[i].first[1]; });
    const Source s = a.source[k];
    const Shape shape = a.shape[k];
    const Grid g(shape);
    const int strips = (g.ct + kStrip - 1) / kStrip;
    const uint32_t at = blockIdx.x - s.first[1];
    const int b = (int)(at / (uint32_t)(g.rt * strips)), rest = (int)(at - (uint32_t)b * (g.rt * strips));
    const int ti = rest / strips, strip = rest - ti * strips;

    static_assert(kMaxSlices <= kPassThreads, "a partial sum a thread");
    Sum sum;
    if (threadIdx.x < s.slices) {
        const Partial p = a.partial[s.at + b * s.slices + threadIdx.x];
        sum.hi = p.hi;
        sum.lo = p.lo;
        sum.wide = p.wide;
    }
    __shared__ float2 found;
    const Sum total = block_total<kPassThreads / 32>(sum);
    if (threadIdx.x == 0) {
        found = factors(total, a.eps);
    }
    __syncthreads();
    const float2 factor = found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tj = strip * kStrip + lane / 8, c = tj * 64 + (lane & 7) * 8;
    if (tj >= g.ct) return;
    uint8_t* const tile = a.tiles + ((int64_t)shape.base + (int64_t)b * g.tiles() + (int64_t)ti * g.ct + tj) * kTileBytes;
    const int64_t lo = (int64_t)g.x_lo() * kTileBytes;
    constexpr int kAhead = kMomentum ? 2 : 4;       // rows a thread has in flight
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += kAhead) {
        Raws<kAhead, kMomentum> raw;
        raw.get(s, b, shape.cols, [&](int i, int& r, int& col) {
            r = ti * 64 + warp + 8 * (i0 + i);
            col = c;
            return r < shape.rows && c < shape.cols;
        });
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = warp + 8 * (i0 + i), row = ti * 64 + r;
            float u[8], kept[8];
            raw.update(a.mu, a.nesterov, s, i, u, kept);
            if (kMomentum && row < shape.rows && c < shape.cols) put8(s.out, b, row, c, shape.cols, kept);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = u[e] * factor.x * factor.y;
            // (a norm that is not a number spreads over the matrix, but not to what lies outside)
            if (row >= shape.rows || c + 8 > shape.cols) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = row < shape.rows && c + e < shape.cols ? u[e] : 0.f;
            }
            uint4 vh, vl;
            split8(u, vh, vl);
            *reinterpret_cast<uint4*>(tile + piece(r, lane & 7)) = vh;
            *reinterpret_cast<uint4*>(tile + lo + piece(r, lane & 7)) = vl;
        }
    }
}

// ---------------------------------------------------------------- the products

struct ProductArgs {
    CUtensorMap map;            // the workspace's tiles as rows of 128 bytes
    int n;
    uint32_t items;             // tiles of the result, of all matrices
    int from;                   // which X is read
    int split;                  // of S, by single CTAs: CTAs (a cluster) an item, each with some of its steps
    float a, b, c, alpha;
    uint8_t* tiles;
    uint32_t* status;
    Shape shape[kTable];
    Result result[kTable];
};

// D tile (i, j) in units of 64 of one matrix, and where its operands are
struct Item {
    int k, b;
    int i, j;                   // first row and column tile
    int steps;                  // of 64 contraction indices
};

// An operand: rows of 64 at `base`, `ld` tiles from one row of tiles to the next.
enum Major { kRowsK, kRowsMn, kSymmetric };
struct Operand {
    int base, lo, ld;
    Major major;
};

// Symmetric matrices are stored on and above the diagonal in blocks of 256 (and read so whatever the
// form of the kernel, as it may change from launch to launch).
constexpr int kSymBlock = 4;                    // tiles of 64 a side

template <int kCtas, int kPhase>
__device__ __forceinline__ Item item_of(const ProductArgs& a, uint32_t t) {
    constexpr int kBlock = 2 * kCtas;           // tiles of 64 a side of a work item
    Item w;
    constexpr int f = is_update(kPhase) ? 1 : 0;
    w.k = element_of(a.n, t, [&](int i) { return a.shape[i].first[f]; });
    const Shape& s = a.shape[w.k];
    const Grid g(s);
    const uint32_t at = t - s.first[f];
    if constexpr (is_update(kPhase)) {
        const int ni = (g.rt + kBlock - 1) / kBlock, nj = (g.ct + kBlock - 1) / kBlock;
        w.b = (int)(at / (uint32_t)(ni * nj));
        const int r = (int)(at - (uint32_t)w.b * (ni * nj));
        // along the smaller side first: its neighbours share X
        w.i = g.wide ? r % ni : r / nj;
        w.j = g.wide ? r / ni : r % nj;
        w.steps = g.mt;
    } else {
        const int nb = (g.mt + kBlock - 1) / kBlock, per = symmetric_items(nb, kCtas);
        w.b = (int)(at / (uint32_t)per);
        int r = (int)(at - (uint32_t)w.b * per);
        // block row i begins with the block of 256 that it is in
        w.i = 0;
        for (int len = nb; r >= len; len = nb - (w.i * kBlock / kSymBlock) * (kSymBlock / kBlock)) {
            r -= len;
            ++w.i;
        }
        w.j = (w.i * kBlock / kSymBlock) * (kSymBlock / kBlock) + r;
        w.steps = g.steps(kPhase);
    }
    w.i *= kBlock;
    w.j *= kBlock;
    return w;
}

template <bool kFull, int kPhase>
__device__ __forceinline__ void operands(const ProductArgs& a, const Item& w, Operand& p, Operand& q, bool& p_lo,
                                         bool& q_lo) {
    const Shape& s = a.shape[w.k];
    const Grid g(s);
    const int at = s.base + w.b * g.tiles();
    const Operand x{at + g.x(a.from), g.x_lo(), g.ct, kRowsK};
    p_lo = q_lo = kFull;
    if constexpr (kPhase == kGram) {
        p = x;
        p.major = g.wide ? kRowsK : kRowsMn;
        q = p;
    } else if constexpr (kPhase == kSquare) {
        p = q = Operand{at + g.s(), g.s_lo(), g.mt, kSymmetric};
    } else {
        const Operand sym{at + g.p(), g.s_lo(), g.mt, kSymmetric};
        p = g.wide ? sym : x;
        q = g.wide ? x : sym;
        if (g.wide) q.major = kRowsMn;
        p_lo = p_lo || !g.wide;
        q_lo = q_lo || g.wide;
    }
}

// Whether the operand's 64 x 64 tiles of block row `first` are K-major at step k.
__device__ __forceinline__ bool k_major(const Operand& o, int first, int k) {
    return o.major == kSymmetric ? first / kSymBlock <= k / kSymBlock : o.major == kRowsK;
}

// ---- PTX of a pair of CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_leader(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// one tile of 64 rows of 128 bytes; bar: a barrier of this CTA or of the pair's first one
template <int kCtas>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, int tile, uint32_t dst, uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(tile * 64), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(tile * 64), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
// until what this thread's stores read (but for the last few), or all they do, is done
template <int kPending = 0>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Where a thread's 64-column blocks of an item go.
struct Place {
    int k, b;
    int rows, cols, m;          // of the matrix, and its smaller side
    int ti, tj, nt, mt;         // tile of the first block; tiles that there are
    int r0, r;                  // in the tile: the warp's first row, this thread's
    int from, to, lo;           // tiles: S, the image that is written, from hi to lo parts
    __device__ __forceinline__ Place(const ProductArgs& a, int phase, const Item& w, int i, int j, int row0, int lane)
        : k(w.k), b(w.b), ti(i), tj(j), r0(row0), r(row0 + lane) {
        const Shape s = a.shape[w.k];
        const Grid g(s);
        const int at = s.base + w.b * g.tiles();
        rows = s.rows;
        cols = s.cols;
        m = min(s.rows, s.cols);
        nt = is_update(phase) ? g.rt : g.mt;
        mt = is_update(phase) ? g.ct : g.mt;
        from = at + g.s();
        to = at + (is_update(phase) ? g.x(1 - a.from) : phase == kGram ? g.s() : g.p());
        lo = is_update(phase) ? g.x_lo() : g.s_lo();
    }
};

// A warp's 32 rows of a tile, as it loads them: piece 32 i + lane of their 4 KB.
struct Lines {
    uint4 v[8];
    __device__ __forceinline__ void get(const uint8_t* tile, const Place& at, int lane) {
        const uint4* p = reinterpret_cast<const uint4*>(tile + 128 * at.r0);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[32 * i + lane];
    }
    __device__ __forceinline__ void put(uint8_t* stage, int lane) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(stage)[32 * i + lane] = v[i];
    }
};
__device__ __forceinline__ const uint8_t* tile_of_s(const ProductArgs& a, const Place& at, int n) {
    return a.tiles + (int64_t)(at.from + at.ti * at.mt + at.tj + n) * kTileBytes;
}

// P from S S (f, scaled): a I + b S + c S S, all scaled, with 8 elements of S.
__device__ __forceinline__ void polynomial8(const ProductArgs& a, const Place& at, int j, int q, const float* s, float* v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = fmaf(a.c, v[e], a.b * s[e]);
        if (at.ti == j && at.r == 8 * q + e && at.ti * 64 + at.r < at.m) v[e] += a.a * kScale;
    }
}

// From full products: S read as it lies, two pieces of hi and lo at a time.
__device__ __forceinline__ void polynomial_full(const ProductArgs& a, const Place& at, int j, float* f) {
    const uint8_t* row = a.tiles + (int64_t)(at.from + at.ti * at.mt + j) * kTileBytes;
    const uint8_t* row_lo = row + (int64_t)at.lo * kTileBytes;
    constexpr int kAhead = 2;
#pragma unroll
    for (int q0 = 0; q0 < 8; q0 += kAhead) {
        uint4 hi[kAhead], lo[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            hi[q] = *reinterpret_cast<const uint4*>(row + piece(at.r, q0 + q));
            lo[q] = *reinterpret_cast<const uint4*>(row_lo + piece(at.r, q0 + q));
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            float s[8];
            join8(hi[q], lo[q], s);
            polynomial8(a, at, j, q0 + q, s, f + 8 * (q0 + q));
        }
    }
}

// From S_hi S_hi: what the low part of S's diagonal (large beside the rest) adds to it comes
// here.  S is loaded in whole lines (its hi part before the accumulators are there) and goes
// through the warp's stage to the threads of its rows.
__device__ __forceinline__ void polynomial_short(const ProductArgs& a, const Place& at, int n, Lines& s, float* f,
                                                 uint8_t* stage, int lane) {
    const int j = at.tj + n;
    const int64_t to_lo = (int64_t)at.lo * kTileBytes;
    auto diagonal = [&](int t, int i) {     // element (i, i) of the low part of diagonal tile t
        const uint8_t* p = a.tiles + (int64_t)(at.from + t * (at.mt + 1)) * kTileBytes + to_lo + piece(i, i >> 3) + (i & 7) * 2;
        return __half2float(*reinterpret_cast<const __half*>(p)) * kUnscale;
    };
    const float own = diagonal(at.ti, at.r);
    const float low[2] = {diagonal(j, lane), diagonal(j, 32 + lane)};   // of columns lane and 32 + lane
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) bulk_wait_read();
    __syncwarp();
    s.put(stage, lane);
    __syncwarp();
    s.get(tile_of_s(a, at, n) + to_lo, at, lane);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float x[8], *v = f + 8 * q;
        join8(*reinterpret_cast<const uint4*>(stage + piece(lane, q)), zero, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = 8 * q + e;
            v[e] = fmaf(own + __shfl_sync(0xffffffffu, low[c / 32], c % 32), x[e], v[e]);
        }
        polynomial8(a, at, j, q, x, v);
    }
    __syncwarp();
    s.put(stage, lane);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float x[8];
        join8(zero, *reinterpret_cast<const uint4*>(stage + piece(lane, q)), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[8 * q + e] = fmaf(a.b, x[e], f[8 * q + e]);
    }
    __syncwarp();
}

// Writes block n of 64 columns (accumulators, which carry 2^24) of this thread's row: to the
// images, or to the result.  kStage: bytes of the warp's stage.
template <bool kFull, int kPhase, int kStage>
__device__ __forceinline__ void write_block(const ProductArgs& a, const Place& at, int n, float* f, Lines& s, int blocks,
                                            uint8_t* stage, int lane) {
    const int j = at.tj + n;
    if (at.ti >= at.nt || j >= at.mt) return;
    if constexpr (kPhase == kResult) {
        // some columns at a time through shared memory, for whole lines
        constexpr int kC = kStage / 128;
        const Result& o = a.result[at.k];
#pragma unroll
        for (int c = 0; c < 64; c += kC) {
            if (j * 64 + c >= at.cols) continue;
            __syncwarp();
#pragma unroll
            for (int q = 0; q < kC / 4; ++q) {
                float4 v;
                v.x = o.beta * (f[c + 4 * q] * (kUnscale * kUnscale));
                v.y = o.beta * (f[c + 4 * q + 1] * (kUnscale * kUnscale));
                v.z = o.beta * (f[c + 4 * q + 2] * (kUnscale * kUnscale));
                v.w = o.beta * (f[c + 4 * q + 3] * (kUnscale * kUnscale));
                *reinterpret_cast<float4*>(stage + staged<kC>(lane, q)) = v;
            }
            __syncwarp();
            write_rows<kC, 4, !kFull>(a.alpha, o, at.b, at.ti * 64 + at.r0, j * 64 + c, at.rows, at.cols, stage, lane);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 64; ++e) f[e] *= kUnscale;
        if constexpr (kPhase == kSquare) {
            if constexpr (kFull) {
                polynomial_full(a, at, j, f);
            } else {
                polynomial_short(a, at, n, s, f, stage, lane);
                if (n + 1 < blocks && j + 1 < at.mt) s.get(tile_of_s(a, at, n + 1), at, lane);
            }
        }
        // 16 rows of a tile are 2 KB in one piece: hi and lo by way of shared memory (16-byte stores
        // of every thread to its own row: 30 us of 138 in S of 2 x 4096 x 4096)
        constexpr int kUnit = 2048;
        constexpr bool kBoth = kStage >= 2 * kUnit;         // hi and lo at once
        uint8_t* dst = a.tiles + (int64_t)(at.to + at.ti * at.mt + j) * kTileBytes + 128 * at.r0;
#pragma unroll 1
        for (int u = 0; u < (kBoth ? 2 : 4); ++u) {
            const int half = kBoth ? u : u >> 1, low = kBoth ? 0 : u & 1;
            if (lane == 0) bulk_wait_read();
            __syncwarp();
            if (lane >> 4 == half) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint4 hi, lo;
                    split8(f + 8 * q, hi, lo);
                    *reinterpret_cast<uint4*>(stage + piece(lane & 15, q)) = low ? lo : hi;
                    if (kBoth) *reinterpret_cast<uint4*>(stage + kUnit + piece(lane & 15, q)) = lo;
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                uint8_t* to = dst + half * kUnit;
                const int64_t to_lo = (int64_t)at.lo * kTileBytes;
                bulk_store(to + (low ? to_lo : 0), stage, kUnit);
                if (kBoth) bulk_store(to + to_lo, stage + kUnit, kUnit);
            }
        }
    }
}

// ---- shared memory: stages of A hi, B hi, then the low parts that are used

constexpr uint32_t kPart = 2 * kTileBytes;              // 128 rows x 64 indices
constexpr uint32_t kRing = 12 * kPart;                  // 192 KB
constexpr int kMaxStages = 6;
constexpr uint32_t kStages = 32768;                     // of the epilogue warps
constexpr uint32_t kBars = kRing + kStages;
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t kSmem = 1024 + kBars + kBarBytes;
static_assert(kSmem <= 232448, "shared memory");

// A warp waits together: warp-uniform control keeps descriptors in uniform registers.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                          uint32_t code) {
    if (__any_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __any_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, status, code));
}

// The tiles that one lane of the TMA warp loads for an item: at step k tile base + k * step, of
// a symmetric operand from step `turn` on the other form of it.
struct Stream {
    int base, step, turn, base2, step2;
    uint32_t dst;               // in the stage
};

// operand o, rows from tile `row` on (of the block from `first` on): its tile number `half`
__device__ __forceinline__ Stream stream_of(const Operand& o, int first, int row, int half, int low, uint32_t dst) {
    const int base = o.base + (low ? o.lo : 0), r = row + half;
    Stream t;
    t.dst = dst;
    // K-major: tile (r, k); MN-major: (k, r); symmetric: MN-major before its own block
    const int k_base = base + r * o.ld, mn_base = base + r;
    t.turn = o.major == kSymmetric ? first / kSymBlock * kSymBlock : 0;
    t.base = o.major == kRowsK ? k_base : mn_base;
    t.step = o.major == kRowsK ? 1 : o.ld;
    t.base2 = o.major == kRowsMn ? mn_base : k_base;
    t.step2 = o.major == kRowsMn ? o.ld : 1;
    return t;
}

// The parts that a cluster's CTAs have of one 128 x 128 block of S (f: 64 columns of a row), added up
// by way of the ring, which is idle then: every CTA gets some rows of all parts, adds them in the order of
// the CTAs and writes them.  128 rows of 512 bytes in all, pieces of 16 bytes in an order that spreads banks.
__device__ __forceinline__ void add_up_split(const ProductArgs& a, const Place& at, uint8_t* ring, int share, int split,
                                             int quad, int part, int lane, const float* f) {
    auto where = [](int row, int q) { return (uint32_t)(row * 512 + ((q ^ (row & 7)) << 4)); };
    const int own = 128 / split, row = 32 * quad + lane;        // rows a CTA; of the block
    cluster_sync();             // every CTA's MMAs are done
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(ring)), "r"(row / own));
#pragma unroll
    for (int q = 0; q < 16; ++q)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + where(share * own + row % own, 16 * part + q)),
                     "f"(f[4 * q]), "f"(f[4 * q + 1]), "f"(f[4 * q + 2]), "f"(f[4 * q + 3])
                     : "memory");
    cluster_sync();
    // pieces of 8 columns: 16 a row
    const int ti0 = at.ti - quad / 2, tj0 = at.tj - part;
    for (int p = (4 * part + quad) * 32 + lane; p < own * 16; p += 256) {
        const int r = p >> 4, c = p & 15;
        float v[8];
        for (int s = 0; s < split; ++s) {
            const float4 x = *reinterpret_cast<const float4*>(ring + where(s * own + r, 2 * c));
            const float4 y = *reinterpret_cast<const float4*>(ring + where(s * own + r, 2 * c + 1));
            const float g[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = s == 0 ? g[e] : v[e] + g[e];
        }
        const int row_of = share * own + r, ti = ti0 + row_of / 64, tj = tj0 + c / 8;
        if (ti >= at.nt || tj >= at.mt) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= kUnscale;
        uint4 hi, lo;
        split8(v, hi, lo);
        uint8_t* dst = a.tiles + (int64_t)(at.to + ti * at.mt + tj) * kTileBytes + piece(row_of & 63, c & 7);
        *reinterpret_cast<uint4*>(dst) = hi;
        *reinterpret_cast<uint4*>(dst + (int64_t)at.lo * kTileBytes) = lo;
    }
}

// kFull: both parts of all operands, accumulators added up in registers every step.  Else the
// accumulators stay in tensor memory for all steps of an item.
//
// Epilogue warps: eight, with 64 or 128 columns a thread and up to 168 registers; for pairs in full
// 16 with 64 columns, as 128 running sums a thread do not fit (2780 cycles a drain, the MMAs take
// 1536): 640 threads, whose 96 registers at launch go 56 to the control warps, 104 to the others.
template <int kCtas, bool kFull>
struct Roles {
    static constexpr bool kMany = kCtas == 2 && kFull;
    static constexpr int kEpiWarps = kMany ? 16 : 8;
    static constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
    static constexpr int kCtl = 56, kEpi = 104, kLaunch = 96;       // registers where kMany
    static_assert(!kMany || kEpiWarp0 * 32 * kCtl + kEpiWarps * 32 * kEpi <= kThreads * kLaunch, "register split");
};

template <int kCtas, bool kFull, int kPhase>
__global__ void __launch_bounds__(Roles<kCtas, kFull>::kThreads, 1) product_kernel(const __grid_constant__ ProductArgs a) {
    using R = Roles<kCtas, kFull>;
    constexpr int kEpiWarps = R::kEpiWarps;
    constexpr int kN = 128 * kCtas;             // columns of the accumulator
    constexpr int kCols = kN * 4 / kEpiWarps;   // of a thread
    constexpr int kStage = kStages / kEpiWarps; // shared memory of an epilogue warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBars);     // [stages] of the leader: all parts landed
    uint64_t* empty = full + kMaxStages;        // [stages] the MMAs that read the stage are done
    uint64_t* zfull = empty + kMaxStages;       // [2]
    uint64_t* zempty = zfull + 2;               // [2] of the leader
    uint64_t* done = zempty + 2;                // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kMaxStages + 5) * 8 + 8 <= kBarBytes, "barriers");
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 2 ? cluster_rank() : 0;
    // one of `split` CTAs that share an item's steps
    constexpr bool kSplits = kCtas == 1 && kPhase == kGram;
    const int split = kSplits ? a.split : 1, share = kSplits && split > 1 ? (int)cluster_rank() : 0;
    // parts a stage: of both operands hi, and lo of both (full) or of one (P X)
    constexpr int parts = kFull ? 4 : is_update(kPhase) ? 3 : 2;
    // steps a stage: with four MMAs a step the control of each would take longer than they do
    // (733 cycles a step for 512 of MMAs)
    constexpr int sub = !kFull && !is_update(kPhase) ? 2 : 1;
    constexpr int stages = 12 / (parts * sub);
    // steps between drains, or of a stage: two in full, but one for items of few (a sum is cut off at every
    // addition: 128 x 1833 with two 1.8 times as far off as fp32 products, with one 1.2)
    constexpr int per_pass = kFull ? 2 : sub;
    auto between = [&](int steps) { return kFull && steps <= 2 ? 1 : per_pass; };
    constexpr uint32_t step_bytes = (uint32_t)parts * kPart, stage_bytes = step_bytes * sub;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int z = 0; z < 2; ++z) {
            mbar_init(&zfull[z], 1);
            mbar_init(&zempty[z], kEpiWarps * kCtas);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (kCtas == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(2 * kN));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(2 * kN));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc_fence_before();
    if constexpr (kCtas == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();

    const uint32_t first = blockIdx.x / (uint32_t)(kCtas * split), stride = gridDim.x / (uint32_t)(kCtas * split);
    auto from_step = [&](const Item& w) { return kSplits ? share_begin(w.steps, share, split) : 0; };
    auto to_step = [&](const Item& w) { return kSplits ? share_begin(w.steps, share + 1, split) : w.steps; };
    if (warp < kEpiWarp0) {
    if constexpr (R::kMany) regs_dec<R::kCtl>();
    if (warp == 0) {
        // ------------- TMA: this CTA's rows of both operands, a lane for each tile of a stage -------------
        asm volatile("fence.proxy.async;" ::: "memory");    // what the kernel before wrote
        const uint32_t ring = smem_u32(smem);
        const int in_step = 2 * parts, mine = lane / in_step, tile_of = lane - mine * in_step;
        uint32_t slot = 0, phase = 0;
        bool reused = false, ok = true;
        for (uint32_t t = first; t < a.items && ok; t += stride) {
            const Item w = item_of<kCtas, kPhase>(a, t);
            Operand p, q;
            bool p_lo, q_lo;
            operands<kFull, kPhase>(a, w, p, q, p_lo, q_lo);
            // tiles 0-3: both operands' hi; behind them the low parts
            const int half = tile_of & 1, which = tile_of >> 1;
            const bool of_p = which == 0 || (which == 2 && p_lo);
            const Operand& o = of_p ? p : q;
            const int block = of_p ? w.i : w.j;
            const Stream m = stream_of(o, block, block + 2 * (int)rank, half, which >= 2,
                                              (uint32_t)mine * step_bytes + (uint32_t)tile_of * kTileBytes);
            const int ke = to_step(w);
            for (int k0 = from_step(w); k0 < ke; k0 += sub) {
                const int k = k0 + mine, here = min(sub, ke - k0);
                const int tile = k < m.turn ? m.base + k * m.step : m.base2 + k * m.step2;
                if (reused && !warp_wait(&empty[slot], phase ^ 1u, abort_flag, a.status, kStatusTimeoutTma)) {
                    ok = false;
                    break;
                }
                if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&full[slot], kCtas * step_bytes * here);
                __syncwarp();
                const uint32_t bar = kCtas == 2 ? in_leader(&full[slot]) : smem_u32(&full[slot]);
                if (mine < here) load_tile<kCtas>(&a.map, tile, ring + slot * stage_bytes + m.dst, bar);
                if (++slot == (uint32_t)stages) {
                    slot = 0;
                    phase ^= 1u;
                    reused = true;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------- MMA: the leader, for both CTAs -------------------------
        if (rank == 0) {
            constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(128 * kCtas >> 4) << 24);
            const uint32_t ring = smem_u32(smem);
            const uint32_t leader = lane == 0 ? 1u : 0u;
            uint32_t slot = 0, phase = 0, z = 0, zphase = 0, zused = 0;
            bool ok = true;
            for (uint32_t t = first; t < a.items && ok; t += stride) {
                const Item w = item_of<kCtas, kPhase>(a, t);
                Operand p, q;
                bool p_lo, q_lo;
                operands<kFull, kPhase>(a, w, p, q, p_lo, q_lo);
                // the MMAs of step k, from the stage at shared-memory address `at`: small terms (low), or hi hi
                auto issue = [&](int k, uint32_t at, uint32_t d, bool small, uint32_t acc) {
                    const bool pk = k_major(p, w.i, k), qk = k_major(q, w.j, k);
                    const uint32_t idesc = kIdesc | (pk ? 0u : 1u << 15) | (qk ? 0u : 1u << 16);
                    const uint32_t p0 = pk ? sdesc128_lo(at) : sdesc128mn_lo(at);
                    const uint32_t q0 = qk ? sdesc128_lo(at + kPart) : sdesc128mn_lo(at + kPart);
                    const uint32_t pstep = pk ? 2u : 128u, qstep = qk ? 2u : 128u;
                    if (!small) {
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk, acc = 1u)
                            mma<kCtas>(d, p0 + kk * pstep, q0 + kk * qstep, idesc, acc, leader);
                        return;
                    }
                    if (kFull || q_lo) {
                        const uint32_t ql = q0 + (((kFull || p_lo ? 2 : 1) * kPart) >> 4);
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk, acc = 1u)
                            mma<kCtas>(d, p0 + kk * pstep, ql + kk * qstep, idesc, acc, leader);
                    }
                    if (kFull || p_lo) {
                        const uint32_t pl = p0 + ((2 * kPart) >> 4);
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk, acc = 1u)
                            mma<kCtas>(d, pl + kk * pstep, q0 + kk * qstep, idesc, acc, leader);
                    }
                };
                auto landed = [&](uint32_t s, uint32_t parity) {
                    const bool here = warp_wait(&full[s], parity, abort_flag, a.status, kStatusTimeoutMma);
                    tc_fence_after();
                    return here;
                };
                auto next = [&](uint32_t& s, uint32_t& parity) {
                    if (++s == (uint32_t)stages) {
                        s = 0;
                        parity ^= 1u;
                    }
                };
                const int kb = from_step(w), ke = to_step(w);
                const int per = between(ke - kb);
                for (int k0 = kb; k0 < ke && ok; k0 += per) {
                    const int here = min(per, ke - k0);
                    if ((kFull || k0 == kb) && ((zused >> z) & 1u)) {
                        if (!(ok = warp_wait(&zempty[z], (zphase >> z) & 1u, abort_flag, a.status, kStatusTimeoutMma))) break;
                        zphase ^= 1u << z;
                    }
                    if (!(ok = landed(slot, phase))) break;
                    const uint32_t d = tmem + z * kN, at = ring + slot * stage_bytes;
                    if constexpr (kFull) {
                        // the small terms of two steps first: a sum loses by its size at every addition
                        issue(k0, at, d, true, 0u);
                        uint32_t slot2 = slot, phase2 = phase;
                        next(slot2, phase2);
                        const uint32_t at2 = ring + slot2 * stage_bytes;
                        if (here == 2) {
                            if (!(ok = landed(slot2, phase2))) break;
                            issue(k0 + 1, at2, d, true, 1u);
                        }
                        issue(k0, at, d, false, 1u);
                        commit<kCtas>(&empty[slot], leader);
                        if (here == 2) {
                            issue(k0 + 1, at2, d, false, 1u);
                            commit<kCtas>(&empty[slot2], leader);
                            slot = slot2;
                            phase = phase2;
                        }
                    } else {
                        for (int k = k0; k < k0 + here; ++k) {
                            const uint32_t from = at + (uint32_t)(k - k0) * step_bytes;
                            if constexpr (is_update(kPhase)) issue(k, from, d, true, k == kb ? 0u : 1u);
                            issue(k, from, d, false, is_update(kPhase) || k > kb ? 1u : 0u);
                        }
                        commit<kCtas>(&empty[slot], leader);
                    }
                    next(slot, phase);
                    if (kFull || k0 + here == ke) {
                        commit<kCtas>(&zfull[z], leader);
                        zused |= 1u << z;
                        z ^= 1u;
                    }
                }
            }
            commit<kCtas>(done, leader);
        }
        if (lane == 0) wait_drain(done, 0, a.status);
    }
    if (split > 1) {        // beside the epilogue's
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    } else {
        if constexpr (R::kMany) regs_inc<R::kEpi>();
        // ------------------------- epilogue -------------------------
        const int quad = warp & 3, part = (warp - kEpiWarp0) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(part * kCols);
        uint8_t* const stage = smem + kRing + (warp - kEpiWarp0) * kStage;
        uint32_t z = 0, zphase = 0;
        auto filled = [&]() {
            const bool here = warp_wait(&zfull[z], (zphase >> z) & 1u, abort_flag, a.status, kStatusTimeoutEpi);
            tc_fence_after();
            return here;
        };
        auto emptied = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kCtas == 2)
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_leader(&zempty[z]))
                                 : "memory");
                else
                    mbar_arrive(&zempty[z]);
            }
            zphase ^= 1u << z;
            z ^= 1u;
        };
        for (uint32_t t = first; t < a.items; t += stride) {
            const Item w = item_of<kCtas, kPhase>(a, t);
            auto place = [&](const Item& w) {
                return Place(a, kPhase, w, w.i + 2 * (int)rank + quad / 2, w.j + part * (kCols / 64), 32 * (quad & 1), lane);
            };
            Lines s;
            if constexpr (kFull) {
                float acc[kCols] = {};
                bool here = true;
                const int of_item = to_step(w) - from_step(w), drains = (of_item + between(of_item) - 1) / between(of_item);
                for (int n = 0; n < drains; ++n) {
                    if (!(here = filled())) break;
                    // columns in flight: all, or what registers there are for
                    constexpr int kAhead = R::kMany ? 32 : 64;
#pragma unroll
                    for (int c = 0; c < kCols; c += kAhead) {
                        uint32_t v[kAhead];
#pragma unroll
                        for (int e = 0; e < kAhead; e += 32) tmem_ld32(lanes + z * kN + c + e, v + e);
                        tmem_ld_wait();
                        if (c + kAhead == kCols) emptied();
#pragma unroll
                        for (int e = 0; e < kAhead; ++e)
                            acc[c + e] = n == 0 ? __uint_as_float(v[e]) : acc[c + e] + __uint_as_float(v[e]);
                    }
                }
                if (!here && split == 1) break;         // (a cluster's barriers wait for all)
#pragma unroll
                for (int e = 0; e < kCols; ++e) acc[e] = uncut(acc[e], of_item <= 2 ? short_of(4) : short_of(8));
                if constexpr (kSplits) {
                    if (split > 1) {
                        add_up_split(a, place(item_of<kCtas, kPhase>(a, t)), smem, share, split, quad, part, lane, acc);
                        continue;
                    }
                }
                const Place at = place(item_of<kCtas, kPhase>(a, t));       // (again: registers are short before)
#pragma unroll
                for (int c = 0; c < kCols; c += 64)
                    write_block<kFull, kPhase, kStage>(a, at, c / 64, acc + c, s, kCols / 64, stage, lane);
            } else {
                const Place at = place(w);
                if (kPhase == kSquare && at.ti < at.nt && at.tj < at.mt) s.get(tile_of_s(a, at, 0), at, lane);
                if (!filled() && split == 1) break;
#pragma unroll
                for (int c = 0; c < kCols; c += 64) {
                    uint32_t v[64];
                    tmem_ld32(lanes + z * kN + c, v);
                    tmem_ld32(lanes + z * kN + c + 32, v + 32);
                    tmem_ld_wait();
                    if (c + 64 == kCols) emptied();
                    float f[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e) f[e] = __uint_as_float(v[e]);
                    if constexpr (kSplits) {
                        if (split > 1) {
                            add_up_split(a, at, smem, share, split, quad, part, lane, f);
                            continue;
                        }
                    }
                    write_block<kFull, kPhase, kStage>(a, at, c / 64, f, s, kCols / 64, stage, lane);
                }
            }
        }
        if (lane == 0) bulk_wait();
    }

    if (*abort_flag) {
        // given up: copies in flight land within microseconds, which nobody waits for any more
        for (int i = 0; i < 100; ++i) __nanosleep(10000);
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (kCtas == 2) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kCtas == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kN));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kN));
    }
}

// ---------------------------------------------------------------- host

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// a list element, or some of its matrices
struct Part {
    int k;
    int64_t b0, count;
};

// Parts of the list that go into one group of launches, from (k, b) on; moves both on.
int next_group(int n, const mttkrp_matrices* like, int& k, int64_t& b, Part* parts, int64_t& tiles) {
    int used = 0;
    tiles = 0;
    while (k < n && used < kTable) {
        const mttkrp_matrices& m = like[k];
        if (m.batch - b <= 0 || !newton_some(m) || newton_is_small(m)) {
            ++k;
            b = 0;
            continue;
        }
        const int64_t per = Grid(Shape{0, (int)m.rows, (int)m.cols, 1, {0, 0}}).tiles();
        int64_t count = std::min(m.batch - b, (kGroupTiles - tiles) / per);
        if (count == 0) {
            if (used > 0) break;
            count = 1;
        }
        parts[used++] = Part{k, b, count};
        tiles += per * count;
        b += count;
        if (b < m.batch) break;         // the group is full
        ++k;
        b = 0;
    }
    return used;
}

// sums of a matrix: of 16 groups of eight columns a thread, more for large ones
int slices_of(const mttkrp_matrices& m) {
    return (int)std::min<int64_t>(cdiv(m.rows * cdiv(m.cols, 8), 16 * kPassThreads), kMaxSlices);
}

size_t partial_bytes(int used, const Part* parts, const mttkrp_matrices* like) {
    int64_t sums = 0;
    for (int i = 0; i < used; ++i) {
        const mttkrp_matrices& m = like[parts[i].k];
        sums += parts[i].count * slices_of(m);
    }
    return (size_t)cdiv(sums * (int64_t)sizeof(Partial), 1024) * 1024;
}

template <int kCtas, bool kFull>
cudaError_t launch_product(int phase, unsigned units, cudaStream_t s, const ProductArgs& p) {     // units: of CTAs or pairs
    const auto kernel = phase == kGram     ? product_kernel<kCtas, kFull, kGram>
                        : phase == kSquare ? product_kernel<kCtas, kFull, kSquare>
                        : phase == kUpdate ? product_kernel<kCtas, kFull, kUpdate>
                                           : product_kernel<kCtas, kFull, kResult>;
    const int cluster = kCtas * (phase == kGram && kCtas == 1 ? p.split : 1);
    return launch_clusters(kernel, units * kCtas, Roles<kCtas, kFull>::kThreads, kSmem, cluster, s, p);
}

// allows a form of the kernels their shared memory
template <int kCtas, bool kFull>
cudaError_t allow() {
    for (const auto kernel : {product_kernel<kCtas, kFull, kGram>, product_kernel<kCtas, kFull, kSquare>,
                              product_kernel<kCtas, kFull, kUpdate>, product_kernel<kCtas, kFull, kResult>}) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        cudaFuncAttributes attr;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kernel);
        // the register split that a kernel asks for waits for ever where its launch has fewer
        if (e == cudaSuccess && Roles<kCtas, kFull>::kMany && attr.numRegs < Roles<kCtas, kFull>::kLaunch)
            e = cudaErrorInvalidConfiguration;
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

struct Device {
    int sms = 0;
};

// allows the kernels their shared memory on the current device, once
cudaError_t device(Device& d) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && known[dev] > 0) {
        d.sms = known[dev];
        return cudaSuccess;
    }
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = allow<1, false>();
    if (e == cudaSuccess) e = allow<1, true>();
    if (e == cudaSuccess) e = allow<2, false>();
    if (e == cudaSuccess) e = allow<2, true>();
    if (e == cudaSuccess && dev < 64) known[dev] = d.sms;
    return e;
}

// Tensor map of the images: rows of 128 bytes, loaded 64 at a time as they are.
bool tile_map(CUtensorMap* map, void* tiles, uint64_t rows) {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 encode = known;
    if (encode == nullptr) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return false;
        known = encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    const cuuint64_t dim[2] = {64, rows}, stride[1] = {128};
    const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, tiles, dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t run_group(const NewtonArgs& a, int used, const Part* parts, int64_t tiles, const Device& d, cudaStream_t s) {
    PassArgs pass;
    ProductArgs p;
    pass.n = p.n = used;
    pass.mu = a.mu;
    pass.nesterov = a.nesterov;
    pass.eps = a.eps;
    pass.partial = static_cast<Partial*>(a.ws);
    pass.tiles = p.tiles = static_cast<uint8_t*>(a.ws) + partial_bytes(used, parts, a.grad);
    p.status = a.status;
    p.alpha = a.alpha;
    bool full = false;          // both parts of every operand
    uint32_t strips = 0;
    int base = 0, sums = 0;
    for (int i = 0; i < used; ++i) {
        const Part& w = parts[i];
        const mttkrp_matrices& m = a.grad[w.k];
        const Shape shape{base, (int)m.rows, (int)m.cols, (int)w.count, {0, 0}};
        const Grid g(shape);
        pass.shape[i] = p.shape[i] = shape;
        Source& u = pass.source[i];
        u.g = store_of(m, w.b0);
        u.m = u.out = Store{nullptr, 0, 0, 0, 0};
        if (a.momentum != nullptr) {
            u.m = store_of(a.momentum[w.k], w.b0);
            u.out = store_of(a.momentum_out[w.k], w.b0);
        }
        u.slices = slices_of(m);
        u.first[0] = (uint32_t)sums;
        u.first[1] = strips;
        u.at = sums;
        sums += (int)(u.slices * w.count);
        strips += (uint32_t)(w.count * g.rt * cdiv(g.ct, kStrip));
        base += (int)(g.tiles() * w.count);
        Result& r = p.result[i];
        r.out = store_of(a.out[w.k], w.b0);
        r.w = a.weight != nullptr ? store_of(a.weight[w.k], w.b0) : Store{nullptr, 0, 0, 0, 0};
        r.beta = a.beta[w.k];
        if (r.out.type != MTTKRP_BF16) full = true;
    }
    if (!tile_map(&p.map, p.tiles, (uint64_t)tiles * 64)) return cudaErrorUnknown;
    cudaError_t e = launch_clusters(a.momentum != nullptr ? squares_kernel<true> : squares_kernel<false>, (unsigned)sums, kPassThreads, 0, 1, s, pass);
    if (e == cudaSuccess) e = launch_clusters(a.momentum != nullptr ? images_kernel<true> : images_kernel<false>, strips, kPassThreads, 0, 1, s, pass);
    for (int step = 0; step < a.steps && e == cudaSuccess; ++step) {
        p.from = step & 1;
        p.a = a.coefficients[3 * step];
        p.b = a.coefficients[3 * step + 1];
        p.c = a.coefficients[3 * step + 2];
        for (int at = kGram; at <= kUpdate && e == cudaSuccess; ++at) {
            const int phase = at == kUpdate && step == a.steps - 1 ? kResult : at;
            const float pair = number_items(p, phase, 2, full, d.sms);
            const int ctas = number_items(p, phase, 1, full, d.sms) <= pair ? 1 : 2;
            if (ctas == 2) number_items(p, phase, 2, full, d.sms);
            const unsigned units = p.split > 1 ? p.items * p.split : std::min<unsigned>(p.items, (unsigned)(d.sms / ctas));
            e = ctas == 2 ? full ? launch_product<2, true>(phase, units, s, p) : launch_product<2, false>(phase, units, s, p)
                          : full ? launch_product<1, true>(phase, units, s, p) : launch_product<1, false>(phase, units, s, p);
        }
    }
    return e;
}

}  // namespace

size_t newton_workspace_bytes(int n, const mttkrp_matrices* like) {
    size_t most = 0;
    Part parts[kTable];
    int k = 0;
    int64_t b = 0, tiles = 0;
    for (int used; (used = next_group(n, like, k, b, parts, tiles)) > 0;)
        most = std::max(most, partial_bytes(used, parts, like) + (size_t)tiles * kTileBytes);
    return most;
}

cudaError_t launch_newton(const NewtonArgs& a, cudaStream_t s) {
    Device d;
    cudaError_t e = device(d);
    if (e == cudaSuccess) e = launch_newton_small(a, d.sms, s);
    Part parts[kTable];
    int k = 0;
    int64_t b = 0, tiles = 0;
    for (int used; e == cudaSuccess && (used = next_group(a.n, a.grad, k, b, parts, tiles)) > 0;)
        e = run_group(a, used, parts, tiles, d, s);
    return e;
}

}  // namespace mk
