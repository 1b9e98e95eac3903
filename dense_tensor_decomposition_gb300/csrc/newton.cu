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
// memory, eight warps drain the other one and write the result.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "launch.cuh"
#include "newton.h"
#include "ptx.cuh"
#include "squares.cuh"
#include "types.cuh"

namespace mk {
namespace {

constexpr int kTable = 32;                  // list elements a group of launches
constexpr int kMaxSlices = 256;             // CTAs a matrix in the passes over U
constexpr uint32_t kTileBytes = 8192;
constexpr int64_t kGroupTiles = (int64_t)4 << 17;   // 4 GB of images a group (one matrix at least)
constexpr float kScale = 4096.f, kUnscale = 1.f / 4096.f;   // of the images

constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;      // 384
constexpr int kPassThreads = 256;

enum Phase { kGram, kSquare, kUpdate };

// Matrices of one list element.  Tiles of one matrix, hi and lo of each: X twice (a step
// reads one and writes the other), S, P.
struct Shape {
    int base;                   // first tile
    int rows, cols, count;
    uint32_t first[2];          // number of the first work item: of S and S S, of P X
};
__host__ __device__ inline int tiles_of(int n) { return (n + 63) / 64; }

struct Grid {
    int rt, ct, mt;             // tiles of 64 along rows, columns and the smaller side
    bool wide;
    __host__ __device__ explicit Grid(const Shape& s)
        : rt(tiles_of(s.rows)), ct(tiles_of(s.cols)), mt(s.rows <= s.cols ? rt : ct), wide(s.rows <= s.cols) {}
    __host__ __device__ int x(int which) const { return 2 * which * rt * ct; }
    __host__ __device__ int x_lo() const { return rt * ct; }
    __host__ __device__ int s() const { return 4 * rt * ct; }
    __host__ __device__ int p() const { return s() + 2 * mt * mt; }
    __host__ __device__ int s_lo() const { return mt * mt; }
    __host__ __device__ int tiles() const { return 4 * (rt * ct + mt * mt); }
};

// Rows of a matrix in its own memory.
struct Store {
    void* data;
    int64_t row, batch;         // strides
    uint8_t type, whole;        // whole: eight elements from a multiple of eight on are aligned to 16 bytes
};

template <typename T>
__device__ __forceinline__ void get8_of(const Store& s, int64_t at, int valid, float* v) {
    const T* p = static_cast<const T*>(s.data) + at;
    if (s.whole && valid >= 8) {
        constexpr int kVec = 16 / sizeof(T);
#pragma unroll
        for (int k = 0; k < 8 / kVec; ++k) {
            const auto w = as_pack<Pack<T, kVec>>(reinterpret_cast<const uint4*>(p)[k]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[k * kVec + e] = to_f32(w.v[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < valid ? to_f32(p[e]) : 0.f;
    }
}
// eight elements of row r from column c on, zeros from `cols` on
__device__ __forceinline__ void get8(const Store& s, int64_t b, int r, int c, int cols, float* v) {
    const int64_t at = b * s.batch + r * s.row + c;
    if (s.type == MTTKRP_F32) get8_of<float>(s, at, cols - c, v);
    else if (s.type == MTTKRP_BF16) get8_of<__nv_bfloat16>(s, at, cols - c, v);
    else get8_of<__half>(s, at, cols - c, v);
}
template <typename T>
__device__ __forceinline__ void put8_of(const Store& s, int64_t at, int valid, const float* v) {
    T* p = static_cast<T*>(s.data) + at;
    if (s.whole && valid >= 8) {
        constexpr int kVec = 16 / sizeof(T);
#pragma unroll
        for (int k = 0; k < 8 / kVec; ++k) {
            Pack<T, kVec> w;
#pragma unroll
            for (int e = 0; e < kVec; ++e) w.v[e] = from_f32<T>(v[k * kVec + e]);
            reinterpret_cast<uint4*>(p)[k] = as_pack<uint4>(w);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = from_f32<T>(v[e]);
    }
}
__device__ __forceinline__ void put8(const Store& s, int64_t b, int r, int c, int cols, const float* v) {
    const int64_t at = b * s.batch + r * s.row + c;
    if (s.type == MTTKRP_F32) put8_of<float>(s, at, cols - c, v);
    else if (s.type == MTTKRP_BF16) put8_of<__nv_bfloat16>(s, at, cols - c, v);
    else put8_of<__half>(s, at, cols - c, v);
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

// byte offset of 16-byte piece c (0-7) of row r in a tile
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// ---------------------------------------------------------------- the passes over U

struct Source {
    Store g, m, out;            // m.data NULL: no momentum
    uint32_t first;             // number of the element's first slice
    int slices;                 // of a matrix
    int at;                     // number of its first partial sum
};

struct PassArgs {
    int n;
    float mu;
    bool nesterov;
    double eps;
    double* partial;
    uint8_t* tiles;
    Shape shape[kTable];
    Source source[kTable];
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

struct Slice {
    int k, b, slice;            // element, matrix, slice of it
    int t0, t1;                 // its tiles
    __device__ explicit Slice(const PassArgs& a) {
        k = element_of(a.n, blockIdx.x, [&](int i) { return a.source[i].first; });
        const Source& s = a.source[k];
        const uint32_t at = blockIdx.x - s.first;
        b = (int)(at / s.slices);
        slice = (int)(at - (uint32_t)b * s.slices);
        const Grid g(a.shape[k]);
        const int64_t tiles = (int64_t)g.rt * g.ct;
        t0 = (int)(tiles * slice / s.slices);
        t1 = (int)(tiles * (slice + 1) / s.slices);
    }
};

// U of eight elements and, where there is momentum, what it becomes
__device__ __forceinline__ void update8(const PassArgs& a, const Source& s, int b, int r, int c, int cols, float* u,
                                        float* kept) {
    get8(s.g, b, r, c, cols, u);
    if (s.m.data != nullptr) {
        get8(s.m, b, r, c, cols, kept);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            kept[e] = fmaf(a.mu, kept[e], u[e]);
            u[e] = a.nesterov ? fmaf(a.mu, kept[e], u[e]) : kept[e];
        }
    }
}

// partial sums of squares, a slice each
__global__ void __launch_bounds__(kPassThreads) squares_kernel(const __grid_constant__ PassArgs a) {
    after_previous();
    const Slice w(a);
    const Source& s = a.source[w.k];
    const Shape& shape = a.shape[w.k];
    const int ct = tiles_of(shape.cols);
    const int tr = threadIdx.x >> 3, tc = (threadIdx.x & 7) * 8;
    Sum sum;
    for (int t = w.t0; t < w.t1; ++t) {
        const int ti = t / ct, c = (t - ti * ct) * 64 + tc;
        float v[16], kept[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = ti * 64 + 32 * h + tr;
            if (r < shape.rows && c < shape.cols) {
                update8(a, s, w.b, r, c, shape.cols, v + 8 * h, kept);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * h + e] = 0.f;
            }
        }
        sum.squares16(v);
    }
    const double total = block_sum<kPassThreads / 32>(sum);
    if (threadIdx.x == 0) a.partial[s.at + w.b * s.slices + w.slice] = total;
}

// the images of X = U / (|U| + eps), zeros behind the last row and column; momentum written
__global__ void __launch_bounds__(kPassThreads) images_kernel(const __grid_constant__ PassArgs a) {
    __shared__ double warp_sum[kPassThreads / 32];
    after_previous();
    const Slice w(a);
    const Source& s = a.source[w.k];
    const Shape& shape = a.shape[w.k];
    const Grid g(shape);
    static_assert(kMaxSlices <= kPassThreads, "a partial sum a thread");
    double norm = threadIdx.x < s.slices ? a.partial[s.at + w.b * s.slices + threadIdx.x] : 0.0;
    for (int o = 16; o > 0; o >>= 1) norm += __shfl_xor_sync(0xFFFFFFFFu, norm, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = norm;
    __syncthreads();
    norm = 0.0;
#pragma unroll
    for (int i = 0; i < kPassThreads / 32; ++i) norm += warp_sum[i];
    const double factor = (double)kScale / (sqrt(norm) + a.eps);
    const bool narrow = factor >= 0x1p-110 && factor <= 0x1p110;     // else (NaN too) the product in fp64
    const float f32 = (float)factor;
    const int tr = threadIdx.x >> 3, tc = threadIdx.x & 7;
    uint8_t* const hi0 = a.tiles + ((int64_t)shape.base + (int64_t)w.b * g.tiles()) * kTileBytes;
    for (int t = w.t0; t < w.t1; ++t) {
        const int ti = t / g.ct, c = (t - ti * g.ct) * 64 + 8 * tc;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 32 * h + tr, row = ti * 64 + r;
            float u[8], kept[8];
            if (row < shape.rows && c < shape.cols) {
                update8(a, s, w.b, row, c, shape.cols, u, kept);
                if (s.m.data != nullptr) put8(s.out, w.b, row, c, shape.cols, kept);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[e] = c + e >= shape.cols ? 0.f : narrow ? u[e] * f32 : (float)((double)u[e] * factor);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = 0.f;
            }
            uint4 vh, vl;
            split8(u, vh, vl);
            uint8_t* at = hi0 + (int64_t)t * kTileBytes + piece(r, tc);
            *reinterpret_cast<uint4*>(at) = vh;
            *reinterpret_cast<uint4*>(at + (int64_t)g.x_lo() * kTileBytes) = vl;
        }
    }
}

// ---------------------------------------------------------------- the products

struct Result {
    Store out, w;               // w.data NULL: alpha is not used
    float beta;
};

struct ProductArgs {
    CUtensorMap map;            // the workspace's tiles as rows of 128 bytes
    int n;
    uint32_t items;             // tiles of the result, of all matrices
    int phase;
    int from;                   // which X is read
    bool full;                  // both parts of every operand
    bool last;                  // of P X: results to `result`
    int chunk;                  // steps of 64 indices between drains
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

template <int kCtas>
__device__ __forceinline__ Item item_of(const ProductArgs& a, uint32_t t) {
    constexpr int kBlock = 2 * kCtas;           // tiles of 64 a side of a work item
    Item w;
    const int f = a.phase == kUpdate ? 1 : 0;
    w.k = element_of(a.n, t, [&](int i) { return a.shape[i].first[f]; });
    const Shape& s = a.shape[w.k];
    const Grid g(s);
    const uint32_t at = t - s.first[f];
    if (a.phase == kUpdate) {
        const int ni = (g.rt + kBlock - 1) / kBlock, nj = (g.ct + kBlock - 1) / kBlock;
        w.b = (int)(at / (uint32_t)(ni * nj));
        const int r = (int)(at - (uint32_t)w.b * (ni * nj));
        // along the smaller side first: its neighbours share X
        w.i = g.wide ? r % ni : r / nj;
        w.j = g.wide ? r / ni : r % nj;
        w.steps = g.mt;
    } else {
        const int nb = (g.mt + kBlock - 1) / kBlock, per = nb * (nb + 1) / 2;
        w.b = (int)(at / (uint32_t)per);
        int r = (int)(at - (uint32_t)w.b * per);
        w.i = 0;
        for (int len = nb; r >= len; --len, ++w.i) r -= len;
        w.j = w.i + r;
        w.steps = a.phase == kSquare ? g.mt : g.wide ? g.ct : g.rt;
    }
    w.i *= kBlock;
    w.j *= kBlock;
    return w;
}

__device__ __forceinline__ void operands(const ProductArgs& a, const Item& w, Operand& p, Operand& q, bool& p_lo,
                                         bool& q_lo) {
    const Shape& s = a.shape[w.k];
    const Grid g(s);
    const int at = s.base + w.b * g.tiles();
    const Operand x{at + g.x(a.from), g.x_lo(), g.ct, kRowsK};
    p_lo = q_lo = a.full;
    if (a.phase == kGram) {
        p = x;
        p.major = g.wide ? kRowsK : kRowsMn;
        q = p;
    } else if (a.phase == kSquare) {
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
template <int kCtas>
__device__ __forceinline__ bool k_major(const Operand& o, int first, int k) {
    constexpr int kBlock = 2 * kCtas;
    return o.major == kSymmetric ? first / kBlock <= k / kBlock : o.major == kRowsK;
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

template <int kCtas>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %3};\n\t"
            "mov.b64 db, {%2, %3};\n\t"
            "setp.ne.b32 p, %5, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n\t}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"((uint32_t)(kDescSw128Hi >> 32)), "r"(idesc), "r"(acc));
    else
        mma_f16_ss(d, a_lo, b_lo, idesc, acc);
}

// arrive on `bar` (of both CTAs) when the MMAs so far are done
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        mma_commit(bar);
}

// ---- shared memory: stages of A hi, B hi, then the low parts that are used

constexpr uint32_t kPart = 2 * kTileBytes;              // 128 rows x 64 indices
constexpr uint32_t kRing = 12 * kPart;                  // 192 KB
constexpr int kMaxStages = 6;
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t kSmem = 1024 + kRing + kBarBytes;
static_assert(kSmem <= 232448, "shared memory");

template <int kCtas>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductArgs a) {
    constexpr int kN = 128 * kCtas;             // columns of the accumulator
    constexpr int kCols = kN / 2;               // of a thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing);     // [stages] of the leader: all parts landed
    uint64_t* empty = full + kMaxStages;        // [stages] the MMAs that read the stage are done
    uint64_t* zfull = empty + kMaxStages;       // [2]
    uint64_t* zempty = zfull + 2;               // [2] of the leader
    uint64_t* done = zempty + 2;                // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kMaxStages + 5) * 8 + 8 <= kBarBytes, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 2 ? cluster_rank() : 0;
    // parts a stage: of both operands hi, and lo of both (full) or of one (P X)
    const int parts = a.full ? 4 : a.phase == kUpdate ? 3 : 2;
    const int stages = 12 / parts;
    const uint32_t stage_bytes = (uint32_t)parts * kPart;

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

    const uint32_t first = blockIdx.x / kCtas, stride = gridDim.x / kCtas;
    if (warp == 0 && lane == 0) {
        // ------------------------- TMA: this CTA's rows of both operands -------------------------
        asm volatile("fence.proxy.async;" ::: "memory");    // what the kernel before wrote
        const uint32_t ring = smem_u32(smem);
        int slot = 0;
        uint32_t phase = 0;
        bool reused = false, ok = true;
        for (uint32_t t = first; t < a.items && ok; t += stride) {
            const Item w = item_of<kCtas>(a, t);
            Operand p, q;
            bool p_lo, q_lo;
            operands(a, w, p, q, p_lo, q_lo);
            const int pi = w.i + 2 * (int)rank, qj = w.j + 2 * (int)rank;
            for (int k = 0; k < w.steps; ++k) {
                if (reused && !wait_bounded(&empty[slot], phase ^ 1u, abort_flag, a.status, kStatusTimeoutTma)) {
                    ok = false;
                    break;
                }
                if (rank == 0) mbar_arrive_expect_tx(&full[slot], kCtas * stage_bytes);
                const uint32_t bar = kCtas == 2 ? in_leader(&full[slot]) : smem_u32(&full[slot]);
                uint32_t dst = ring + (uint32_t)slot * stage_bytes;
                const bool pk = k_major<kCtas>(p, w.i, k), qk = k_major<kCtas>(q, w.j, k);
                const int p0 = p.base + (pk ? pi * p.ld + k : k * p.ld + pi), ps = pk ? p.ld : 1;
                const int q0 = q.base + (qk ? qj * q.ld + k : k * q.ld + qj), qs = qk ? q.ld : 1;
                load_tile<kCtas>(&a.map, p0, dst, bar);
                load_tile<kCtas>(&a.map, p0 + ps, dst + kTileBytes, bar);
                load_tile<kCtas>(&a.map, q0, dst + kPart, bar);
                load_tile<kCtas>(&a.map, q0 + qs, dst + kPart + kTileBytes, bar);
                dst += 2 * kPart;
                if (p_lo) {
                    load_tile<kCtas>(&a.map, p0 + p.lo, dst, bar);
                    load_tile<kCtas>(&a.map, p0 + p.lo + ps, dst + kTileBytes, bar);
                    dst += kPart;
                }
                if (q_lo) {
                    load_tile<kCtas>(&a.map, q0 + q.lo, dst, bar);
                    load_tile<kCtas>(&a.map, q0 + q.lo + qs, dst + kTileBytes, bar);
                }
                if (++slot == stages) {
                    slot = 0;
                    phase ^= 1u;
                    reused = true;
                }
            }
        }
    } else if (warp == 1 && lane == 0) {
        // ------------------------- MMA: the leader, for both CTAs -------------------------
        if (rank == 0) {
            constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(128 * kCtas >> 4) << 24);
            const uint32_t ring = smem_u32(smem);
            int slot = 0, z = 0;
            uint32_t phase = 0, zphase = 0, zused = 0;
            bool ok = true;
            for (uint32_t t = first; t < a.items && ok; t += stride) {
                const Item w = item_of<kCtas>(a, t);
                Operand p, q;
                bool p_lo, q_lo;
                operands(a, w, p, q, p_lo, q_lo);
                int in_chunk = 0;
                for (int k = 0; k < w.steps; ++k) {
                    if (in_chunk == 0 && ((zused >> z) & 1u)) {
                        if (!wait_bounded(&zempty[z], (zphase >> z) & 1u, abort_flag, a.status, kStatusTimeoutMma)) {
                            ok = false;
                            break;
                        }
                        zphase ^= 1u << z;
                        tc_fence_after();
                    }
                    if (!wait_bounded(&full[slot], phase, abort_flag, a.status, kStatusTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool pk = k_major<kCtas>(p, w.i, k), qk = k_major<kCtas>(q, w.j, k);
                    const uint32_t idesc = kIdesc | (pk ? 0u : 1u << 15) | (qk ? 0u : 1u << 16);
                    const uint32_t at = ring + (uint32_t)slot * stage_bytes;
                    const uint32_t p0 = pk ? sdesc128_lo(at) : sdesc128mn_lo(at);
                    const uint32_t q0 = qk ? sdesc128_lo(at + kPart) : sdesc128mn_lo(at + kPart);
                    const uint32_t pl = p0 + ((2 * kPart) >> 4), ql = q0 + (((p_lo ? 2 : 1) * kPart) >> 4);
                    const uint32_t pstep = pk ? 2u : 128u, qstep = qk ? 2u : 128u;
                    const uint32_t d = tmem + (uint32_t)(z * kN);
                    // the small terms first: a sum loses by its size at every addition
                    uint32_t acc = in_chunk == 0 ? 0u : 1u;
                    if (q_lo) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk, acc = 1u) mma<kCtas>(d, p0 + kk * pstep, ql + kk * qstep, idesc, acc);
                    }
                    if (p_lo) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk, acc = 1u) mma<kCtas>(d, pl + kk * pstep, q0 + kk * qstep, idesc, acc);
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk, acc = 1u) mma<kCtas>(d, p0 + kk * pstep, q0 + kk * qstep, idesc, acc);
                    commit<kCtas>(&empty[slot]);
                    if (++in_chunk == a.chunk || k == w.steps - 1) {
                        commit<kCtas>(&zfull[z]);
                        zused |= 1u << z;
                        z ^= 1;
                        in_chunk = 0;
                    }
                    if (++slot == stages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            commit<kCtas>(done);
        }
        wait_drain(done, 0, a.status);
    } else if (warp >= kEpiWarp0) {
        // ------------------------- epilogue: eight warps -------------------------
        const int quad = warp & 3, part = (warp - kEpiWarp0) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(part * kCols);
        int z = 0;
        uint32_t zphase = 0;
        bool ok = true;
        for (uint32_t t = first; t < a.items && ok; t += stride) {
            const Item w = item_of<kCtas>(a, t);
            float acc[kCols];
            const int chunks = (w.steps + a.chunk - 1) / a.chunk;
            for (int n = 0; n < chunks; ++n) {
                bool here = true;
                if (lane == 0)
                    here = wait_bounded(&zfull[z], (zphase >> z) & 1u, abort_flag, a.status, kStatusTimeoutEpi);
                if (!__shfl_sync(0xffffffffu, here ? 1 : 0, 0)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t from = lanes + (uint32_t)(z * kN);
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(from + c, v);
                    tmem_ld_wait();
                    if (n == 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) acc[c + e] = __uint_as_float(v[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) acc[c + e] += __uint_as_float(v[e]);
                    }
                }
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
                z ^= 1;
            }
            if (!ok) break;
            // this thread's row and columns of the result
            const Shape& s = a.shape[w.k];
            const Grid g(s);
            const int ti = w.i + 2 * (int)rank + quad / 2, r = 32 * (quad & 1) + lane;
            const int tj = w.j + part * (kCols / 64);
            const int nt = a.phase == kUpdate ? g.rt : g.mt, mt = a.phase == kUpdate ? g.ct : g.mt;
            if (ti >= nt) continue;
            const int at = s.base + w.b * g.tiles();
            if (a.phase == kUpdate && a.last) {
                const Result& o = a.result[w.k];
                const int row = ti * 64 + r;
#pragma unroll
                for (int c = 0; c < kCols; c += 8) {
                    const int col = tj * 64 + c;
                    if (row >= s.rows || col >= s.cols) continue;
                    float v[8];
                    if (o.w.data != nullptr) {
                        get8(o.w, w.b, row, col, s.cols, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = fmaf(a.alpha, v[e], o.beta * (acc[c + e] * (kUnscale * kUnscale)));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = o.beta * (acc[c + e] * (kUnscale * kUnscale));
                    }
                    put8(o.out, w.b, row, col, s.cols, v);
                }
                continue;
            }
            // images: accumulators carry 2^24
            const int to = at + (a.phase == kUpdate ? g.x(1 - a.from) : a.phase == kGram ? g.s() : g.p());
            const int64_t lo = (int64_t)(a.phase == kUpdate ? g.x_lo() : g.s_lo()) * kTileBytes;
            const int64_t back = (int64_t)(g.p() - g.s()) * kTileBytes;     // from P to S
            const bool mend = a.phase == kSquare && !a.full;
            // the low part of S's element (i, i), times 2^12
            auto diagonal = [&](int i) {
                const int at_tile = at + g.s() + g.s_lo() + (i >> 6) * (mt + 1);
                const uint8_t* p = a.tiles + (int64_t)at_tile * kTileBytes + piece(i & 63, (i & 63) >> 3) + (i & 7) * 2;
                return __half2float(*reinterpret_cast<const __half*>(p));
            };
            const float own = mend ? diagonal(ti * 64 + r) * kUnscale : 0.f;
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
                const int j = tj + c / 64;
                if (j >= mt) continue;
                uint8_t* hi_at = a.tiles + (int64_t)(to + ti * mt + j) * kTileBytes + piece(r, (c % 64) / 8);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = acc[c + e] * kUnscale;
                if (a.phase == kSquare) {
                    float sv[8];
                    const uint4 shi = *reinterpret_cast<const uint4*>(hi_at - back);
                    join8(shi, *reinterpret_cast<const uint4*>(hi_at - back + lo), sv);
                    if (mend) {
                        float lead[8];
                        join8(shi, make_uint4(0u, 0u, 0u, 0u), lead);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = fmaf(own + diagonal(j * 64 + c % 64 + e) * kUnscale, lead[e], v[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = fmaf(a.c, v[e], a.b * sv[e]);
                        const int row = ti * 64 + r;
                        if (row == j * 64 + c % 64 + e && row < (g.wide ? s.rows : s.cols)) v[e] += a.a * kScale;
                    }
                }
                uint4 hi, low;
                split8(v, hi, low);
                *reinterpret_cast<uint4*>(hi_at) = hi;
                *reinterpret_cast<uint4*>(hi_at + lo) = low;
            }
        }
    }

    if (*abort_flag) {
        // given up: copies in flight land within microseconds, which nobody waits for any more
        for (int i = 0; i < 100; ++i) __nanosleep(10000);
    }
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
        if (m.batch - b <= 0 || m.rows == 0 || m.cols == 0) {
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

// CTAs of the passes over U for one matrix: a tile each, but for large ones
int slices_of(int64_t tiles) { return (int)std::min<int64_t>(tiles, kMaxSlices); }

size_t partial_bytes(int used, const Part* parts, const mttkrp_matrices* like) {
    int64_t sums = 0;
    for (int i = 0; i < used; ++i) {
        const mttkrp_matrices& m = like[parts[i].k];
        sums += parts[i].count * slices_of(cdiv(m.rows, 64) * cdiv(m.cols, 64));
    }
    return (size_t)cdiv(sums * 8, 1024) * 1024;
}

Store store_of(const mttkrp_matrices& m, int64_t b0) {
    const int64_t elem = m.type == MTTKRP_F32 ? 4 : 2, row = m.rows > 1 ? m.row_stride : 0, batch = m.batch > 1 ? m.batch_stride : 0;
    Store s;
    s.data = static_cast<uint8_t*>(m.data) + b0 * batch * elem;
    s.row = row;
    s.batch = batch;
    s.type = (uint8_t)m.type;
    s.whole = (reinterpret_cast<uintptr_t>(m.data) % 16 == 0 && row * elem % 16 == 0 && batch * elem % 16 == 0) ? 1 : 0;
    return s;
}

template <typename K, typename A>
cudaError_t launch(K kernel, unsigned blocks, unsigned threads, size_t smem, int cluster, cudaStream_t s, const A& args) {
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
    if (e == cudaSuccess) e = cudaFuncSetAttribute(product_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(product_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess && dev < 64) known[dev] = d.sms;
    return e;
}

// Work items of the products with tiles of 64 x kBlock a side, into the shapes.
void count_items(ProductArgs& p, int block, uint32_t* items) {
    items[0] = items[1] = 0;
    for (int i = 0; i < p.n; ++i) {
        Shape& s = p.shape[i];
        const Grid g(s);
        const int64_t nb = cdiv(g.mt, block);
        s.first[0] = items[0];
        s.first[1] = items[1];
        items[0] += (uint32_t)(s.count * (nb * (nb + 1) / 2));
        items[1] += (uint32_t)(s.count * cdiv(g.rt, block) * cdiv(g.ct, block));
    }
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
    pass.partial = static_cast<double*>(a.ws);
    pass.tiles = p.tiles = static_cast<uint8_t*>(a.ws) + partial_bytes(used, parts, a.grad);
    p.status = a.status;
    p.alpha = a.alpha;
    p.full = false;
    uint32_t blocks = 0;
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
        u.first = blocks;
        u.slices = slices_of((int64_t)g.rt * g.ct);
        u.at = sums;
        blocks += (uint32_t)(u.slices * w.count);
        sums += (int)(u.slices * w.count);
        base += (int)(g.tiles() * w.count);
        Result& r = p.result[i];
        r.out = store_of(a.out[w.k], w.b0);
        r.w = a.weight != nullptr ? store_of(a.weight[w.k], w.b0) : Store{nullptr, 0, 0, 0, 0};
        r.beta = a.beta[w.k];
        if (r.out.type != MTTKRP_BF16) p.full = true;
    }
    if (!tile_map(&p.map, p.tiles, (uint64_t)tiles * 64)) return cudaErrorUnknown;
    cudaError_t e = launch(squares_kernel, blocks, kPassThreads, 0, 1, s, pass);
    if (e == cudaSuccess) e = launch(images_kernel, blocks, kPassThreads, 0, 1, s, pass);
    const int ctas = 1;
    uint32_t items[2];
    count_items(p, 2 * ctas, items);
    for (int step = 0; step < a.steps && e == cudaSuccess; ++step) {
        p.from = step & 1;
        p.last = step == a.steps - 1;
        p.a = a.coefficients[3 * step];
        p.b = a.coefficients[3 * step + 1];
        p.c = a.coefficients[3 * step + 2];
        p.chunk = p.full ? 1 : 8;
        for (int phase = kGram; phase <= kUpdate && e == cudaSuccess; ++phase) {
            p.phase = phase;
            p.items = items[phase == kUpdate ? 1 : 0];
            const unsigned units = std::min<unsigned>(p.items, (unsigned)(d.sms / ctas));
            e = ctas == 2 ? launch(product_kernel<2>, units * 2, kThreads, kSmem, 2, s, p)
                          : launch(product_kernel<1>, units, kThreads, kSmem, 1, s, p);
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
    Part parts[kTable];
    int k = 0;
    int64_t b = 0, tiles = 0;
    for (int used; e == cudaSuccess && (used = next_group(a.n, a.grad, k, b, parts, tiles)) > 0;)
        e = run_group(a, used, parts, tiles, d, s);
    return e;
}

}  // namespace mk
