// Lookup of a table's rows, and its gradient by sorted tokens:
//   out[t, :] = scale * table[idx[t], :],
//   out[v, :] (+)= scale * sum over t with idx[t] = v of grad[t, :].
#include <cmath>

#include "sums.cuh"

namespace mk {
namespace {

// ---------------------------------------------------------------- lookup

// Bound by memory (the rows met, and the result).  L lanes take one part of K tokens'
// rows: U vectors of VEC elements each, L vectors apart.  The tokens' indices, then all
// vectors are loaded before the first is stored.
template <typename T, int VEC, int U, int K>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const __grid_constant__ LookupArgs a, int log2L) {
    using P = Pack<T, VEC>;
    using B = typename Bits<sizeof(P)>::type;
    after_previous();
    const int lane = threadIdx.x & ((1 << log2L) - 1);
    const int64_t t0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2L) * K;
    const int step = VEC << log2L;
    const int c0 = (int)blockIdx.y * U * step + lane * VEC;
    const int width = (int)a.width;
    int64_t v[K];
    B x[K][U];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = t0 + k < a.index.n ? index_at(a.index, t0 + k, 0) : -1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (v[k] < 0 || v[k] >= a.index.rows[0]) v[k] = -1;
        const T* src = static_cast<const T*>(a.table) + v[k] * a.table_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v[k] >= 0 && c0 + u * step < width) x[k][u] = *reinterpret_cast<const B*>(src + c0 + u * step);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (t0 + k >= a.index.n) break;
        T* dst = static_cast<T*>(a.out) + (t0 + k) * a.out_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + u * step >= width) break;
            P p = as_pack<P>(x[k][u]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.v[e] = from_f32<T>(v[k] >= 0 ? a.scale * to_f32(p.v[e]) : 0.f);
            *reinterpret_cast<B*>(dst + c0 + u * step) = as_pack<B>(p);
        }
    }
}

// Narrow rows at other offsets, in pieces of VEC elements: the result as one array, 4
// bytes of it a thread and step, whatever rows they are of.  Its rows have no gaps, and it
// starts at a multiple of 4 bytes.  (Read and write, two tokens a row of 400 MB, this way
// and by lookup_pieces: 17 fp32 columns 3.6 and 2.0 TB/s, 33 4.2 and 3.6, 65 4.8 and 4.9,
// 162 5.0 and 6.1; of 16 bits 17 columns 2.0 and 1.0, 65 2.5 and 2.6, 162 3.2 and 5.2.)
// What stands for a row outside the table, `none`, is the zero whose product with the
// scale is +0; scales that are not finite have none and are not taken.  (A bit a piece
// that says which are inside takes fp32 from 32 registers to 46: 17 columns 610 us
// instead of 442.)
constexpr int kFlatSteps = 8;
constexpr int64_t kFlatPieces = 64;         // at most

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) lookup_flat_kernel(const __grid_constant__ LookupArgs a, uint32_t inverse,
                                                               typename Bits<sizeof(T)>::type none) {
    constexpr int S = 4 / sizeof(T) / VEC, kSpan = kThreads * kFlatSteps * S;     // pieces of a store, of a CTA
    using P = Pack<T, VEC>;
    after_previous();
    const uint32_t width = (uint32_t)(a.width / VEC);
    const int64_t total = a.index.n * width, base = (int64_t)blockIdx.x * kSpan;
    const int64_t t0 = base / width;
    const uint32_t rest = (uint32_t)(base - t0 * width);
    Pack<P, S> x[kFlatSteps];
#pragma unroll
    for (int u = 0; u < kFlatSteps; ++u) {
        const uint32_t at = (u * kThreads + threadIdx.x) * S;
#pragma unroll
        for (int e = 0; e < S; ++e) {
            // both are below 2^13, so the quotient is exact: inverse is 2^32 / width rounded up
            const uint32_t i = rest + at + e, r = width == 1 ? i : __umulhi(i, inverse);
            const int64_t v = base + at + e < total ? index_at(a.index, t0 + r, 0) : -1;
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[u].v[e].v[k] = as_pack<T>(none);
            if (v >= 0 && v < a.index.rows[0])
                x[u].v[e] = *reinterpret_cast<const P*>(static_cast<const T*>(a.table) + v * a.table_stride +
                                                        (i - r * width) * VEC);
        }
    }
    P* out = static_cast<P*>(a.out) + base;
#pragma unroll
    for (int u = 0; u < kFlatSteps; ++u) {
        const uint32_t at = (u * kThreads + threadIdx.x) * S;
#pragma unroll
        for (int e = 0; e < S; ++e)
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[u].v[e].v[k] = from_f32<T>(a.scale * to_f32(x[u].v[e].v[k]));
        if (base + at + S <= total) *reinterpret_cast<Pack<P, S>*>(out + at) = x[u];
        else if (base + at < total) out[at] = x[u].v[0];
    }
}

// lanes for a row of `items` loads: a power of two, at most a warp
int log2_lanes(int64_t items) {
    int l = 0;
    while (l < 5 && ((int64_t)1 << l) < items) ++l;
    return l;
}

// `lanes` (a power of two's logarithm) for a part of a row
template <typename T, int VEC, int U, int K>
cudaError_t lookup_by(const LookupArgs& a, int lanes, cudaStream_t s) {
    const dim3 grid((unsigned)cdiv(cdiv(a.index.n, K) << lanes, kThreads),
                    (unsigned)cdiv(a.width, (int64_t)(VEC * U) << lanes));
    return launch_early(lookup_kernel<T, VEC, U, K>, grid, kThreads, 0, s, a, lanes);
}

// Rows of 16-byte vectors, 64 bytes of them a thread.  Rows of 1 KB and more go in parts
// of 512 bytes: the grid takes all tokens' first parts, then the next, so that of a table
// larger than L2 a part's columns stay there for the rows met again.  But a part's ends
// must not share their 32 bytes with the next part's, a write of its own: such rows go in
// one part where 128 lanes can have it.  (Read and write, two tokens a row of 400 MB: 2048
// fp32 columns 9.1 TB/s in parts of 512 bytes, 8.0 of 2 KB, 7.2 in one; 1004 columns 6.0
// in parts, 7.1 in one; 200 columns 6.2 and 6.9; 64 columns in 16 lanes of one load each
// 4.4, in 4 of four loads 7.2.)
template <typename T>
cudaError_t lookup_vectors(const LookupArgs& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T), U = 4, kMost = 7;
    const int64_t vecs = cdiv(a.width, kVec);
    if (vecs <= 4) return lookup_by<T, kVec, 1, 4>(a, log2_lanes(vecs), s);
    if (vecs <= 8) return lookup_by<T, kVec, 2, 2>(a, 2, s);
    int lanes = 2;
    while (lanes < kMost && ((int64_t)U << lanes) < vecs) ++lanes;
    const bool apart = (vecs | a.out_stride / kVec) % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    if (((int64_t)U << lanes) < vecs || (apart && vecs >= 64)) lanes = 3;
    return lookup_by<T, kVec, U, 1>(a, lanes, s);
}

// Rows at other offsets, in pieces of VEC elements: 16 of them a thread, by 8 lanes at
// least.  A part's ends share their 32 bytes with the next part's, a write of its own: so in
// one part where 128 lanes can have it, else in parts of 32 lanes (read and write, two
// tokens a row of 400 MB: 515 fp32 columns 5.0 TB/s in parts of 512 columns, 5.9 in one;
// 1001 columns 6.7 and 7.1; 9001 columns 7.6 in parts of 512 columns, 6.5 in parts of 4096).
template <typename T, int VEC>
cudaError_t lookup_pieces(const LookupArgs& a, cudaStream_t s) {
    constexpr int U = 16, kMost = 7;
    const int64_t width = a.width / VEC;
    if (width <= kFlatPieces && a.out_stride == a.width && reinterpret_cast<uintptr_t>(a.out) % 4 == 0 &&
        std::isfinite(a.scale)) {
        constexpr int64_t kSpan = kThreads * kFlatSteps * (4 / sizeof(T) / VEC);
        const uint32_t inverse = (uint32_t)((((uint64_t)1 << 32) + width - 1) / width);
        using B = typename Bits<sizeof(T)>::type;
        const B none = std::signbit(a.scale) ? (B)1 << (8 * sizeof(T) - 1) : 0;
        return launch_early(lookup_flat_kernel<T, VEC>, (unsigned)cdiv(a.index.n * width, kSpan), kThreads, 0, s, a,
                            inverse, none);
    }
    int lanes = width > 4 ? 3 : log2_lanes(width);
    while (lanes < kMost && ((int64_t)U << lanes) < width) ++lanes;
    if (((int64_t)U << lanes) < width) lanes = 5;
    return lookup_by<T, VEC, U, 2>(a, lanes, s);
}

// the widest vectors that the rows' starts and width allow
template <typename T>
cudaError_t lookup(const LookupArgs& a, cudaStream_t s) {
    constexpr int e = sizeof(T);
    const size_t all = reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.out) |
                       (a.table_stride * e) | (a.out_stride * e) | (a.width * e);
    if (all % 16 == 0) return lookup_vectors<T>(a, s);
    if (all % 4 == 0) return lookup_pieces<T, 4 / e>(a, s);
    return lookup_pieces<T, 1>(a, s);
}

// ---------------------------------------------------------------- gradient

// the gradient's rows, kB of them loaded at a time
template <typename T, int VEC, int B>
struct Grad {
    template <typename List>
    struct Terms {
        static constexpr int kB = B;
        static constexpr bool kAllLanes = false;
        const TermsOf& of;
        const List& list;
        const int p1;
        const int64_t col;
        uint32_t keys[B];
        using P = Pack<T, VEC>;
        using Raw = typename Bits<sizeof(P)>::type;
        Raw x[B];
        __device__ __forceinline__ Terms(const TermsOf& of, const List& list, int, int p1, int64_t col)
            : of(of), list(list), p1(p1), col(col) {}
        __device__ __forceinline__ void load(int p) {
    #pragma unroll
            for (int j = 0; j < B; ++j) {
                const uint2 entry = list(p + j < p1 ? p + j : p);
                keys[j] = entry.x;
                x[j] = *reinterpret_cast<const Raw*>(static_cast<const T*>(of.a.grad) +
                                                     (int64_t)entry.y * of.a.grad_stride + col);
            }
        }
        __device__ __forceinline__ uint32_t key(int j) const { return keys[j]; }
        __device__ __forceinline__ void add(int j, float* acc) const {
            const P v = as_pack<P>(x[j]);
    #pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += to_f32(v.v[e]);
        }
    };
};

// Rows of 16-byte vectors: each of kThreads threads keeps the next kSlots tokens' vectors
// of its columns on their way into shared memory, which takes no registers and, as only the
// thread itself reads them, no barrier.  (With copies of 4 bytes this is slower than plain
// loads: 33271 x 4034 fp32 tokens, 285 us against 261.)
template <typename T, int kThreads, int kSlots>
struct Ring {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int kBytes = 16 * kSlots;

    template <typename List>
    struct Terms {
        static constexpr int kB = 4;
        static constexpr bool kAllLanes = false;
        const TermsOf& of;
        const List& list;
        const int p0, p1;
        const T* at;                // the lane's columns of row 0
        uint32_t ring;              // shared-memory address of the thread's slot 0
        uint32_t keys[kB];
        Pack<T, kVec> x[kB];
        __device__ __forceinline__ Terms(const TermsOf& of, const List& list, int p0, int p1, int64_t col)
            : of(of), list(list), p0(p0), p1(p1), at(static_cast<const T*>(of.a.grad) + col) {
            extern __shared__ float4 ring_smem[];
            ring = (uint32_t)__cvta_generic_to_shared(ring_smem + threadIdx.x);
#pragma unroll
            for (int k = 0; k < kSlots - kB; k += kB) copy(p0 + k);
        }
        __device__ __forceinline__ uint32_t slot(int p) const {
            return ring + ((p - p0) & (kSlots - 1)) * (kThreads * 16);
        }
        // tokens p .. p + kB towards their slots; a group of copies even where there are none
        __device__ __forceinline__ void copy(int p) {
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                if (p + j < p1) {
                    const T* src = at + (int64_t)list(p + j).y * of.a.grad_stride;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(slot(p + j)), "l"(src) : "memory");
                }
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        }
        __device__ __forceinline__ void load(int p) {
            copy(p + kSlots - kB);
            asm volatile("cp.async.wait_group %0;\n" ::"n"(kSlots / kB - 1) : "memory");
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                keys[j] = list(p + j < p1 ? p + j : p).x;
                uint32_t* w = reinterpret_cast<uint32_t*>(x[j].v);
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(slot(p + j))
                             : "memory");
            }
        }
        __device__ __forceinline__ uint32_t key(int j) const { return keys[j]; }
        __device__ __forceinline__ void add(int j, float* acc) const {
#pragma unroll
            for (int e = 0; e < kVec; ++e) acc[e] += to_f32(x[j].v[e]);
        }
    };
};

// rows in vectors of 16 bytes, of two elements or of one, as all starts allow
template <typename T, typename TO>
cudaError_t lookup_grad(const RowSumArgs& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    const size_t from = reinterpret_cast<uintptr_t>(a.grad) | (a.grad_stride * sizeof(T)) | (a.width * sizeof(T));
    const size_t to = reinterpret_cast<uintptr_t>(a.out[0]) | (a.out_stride * sizeof(TO));
    auto vectors_of = [&](size_t v) { return from % (v * sizeof(T)) == 0 && to % (v * sizeof(TO)) == 0; };
    if (vectors_of(kVec))
        return sums_by<TO, kVec, Ring<T, kSumThreads, 8>::template Terms, Ring<T, kSumThreads, 8>::kBytes,
                       Ring<T, kThreads, 16>::template Terms, Ring<T, kThreads, 16>::kBytes>(a, s);
    if (vectors_of(2))
        return sums_by<TO, 2, Grad<T, 2, 8>::template Terms, 0, Grad<T, 2, 8>::template Terms, 0>(a, s);
    return sums_by<TO, 1, Grad<T, 1, 8>::template Terms, 0, Grad<T, 1, 12>::template Terms, 0>(a, s);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, int type, cudaStream_t s) {
    if (a.index.n == 0) return cudaSuccess;
    if (type == MTTKRP_F32) return lookup<float>(a, s);
    if (type == MTTKRP_BF16) return lookup<__nv_bfloat16>(a, s);
    return lookup<__half>(a, s);
}

size_t lookup_grad_workspace_bytes(const IndexArgs& index, int64_t width) {
    if (always_owned(index, width)) return 0;
    return plan_sort(index, sizeof(uint2), kSms).total() + part_bytes(index, width);
}

cudaError_t launch_lookup_grad(const RowSumArgs& a, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if (a.type == MTTKRP_F32) return lookup_grad<float, float>(a, s);
    if (a.type == MTTKRP_BF16)
        return a.out_type == MTTKRP_F32 ? lookup_grad<bf16, float>(a, s) : lookup_grad<bf16, bf16>(a, s);
    return a.out_type == MTTKRP_F32 ? lookup_grad<__half, float>(a, s) : lookup_grad<__half, __half>(a, s);
}

}  // namespace mk
