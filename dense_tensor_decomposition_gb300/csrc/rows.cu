// Lookup of a table's rows, and its gradient by sorted tokens:
//   out[t, :] = scale * table[idx[t], :],
//   out[v, :] (+)= scale * sum over t with idx[t] = v of grad[t, :].
#include "sums.cuh"

namespace mk {
namespace {

// ---------------------------------------------------------------- lookup

// Bound by memory (the rows met, and the result).  L lanes take one part of one
// row: U vectors of VEC elements each, L vectors apart, all loaded before the first
// is stored.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(kThreads) lookup_kernel(LookupArgs a, int log2L) {
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x & ((1 << log2L) - 1);
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2L;
    if (t >= a.index.n) return;
    const int step = VEC << log2L;
    const int c0 = (int)blockIdx.y * U * step + lane * VEC;
    const int width = (int)a.width;
    const int64_t v = index_at(a.index, t, 0);
    const bool inside = v >= 0 && v < a.index.rows[0];
    P x[U];
    if (inside) {
        const T* src = static_cast<const T*>(a.table) + v * a.table_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * step < width) x[u] = *reinterpret_cast<const P*>(src + c0 + u * step);
    }
    T* dst = static_cast<T*>(a.out) + t * a.out_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (c0 + u * step >= width) break;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[u].v[e] = from_f32<T>(inside ? a.scale * to_f32(x[u].v[e]) : 0.f);
        *reinterpret_cast<P*>(dst + c0 + u * step) = x[u];
    }
}

// lanes for a row of `items` loads: a power of two, at most a warp
int log2_lanes(int64_t items) {
    int l = 0;
    while (l < 5 && ((int64_t)1 << l) < items) ++l;
    return l;
}

template <typename T, int VEC, int U>
cudaError_t lookup_by(const LookupArgs& a, cudaStream_t s) {
    const int l = log2_lanes(cdiv(a.width, VEC));
    const dim3 grid((unsigned)cdiv(a.index.n << l, kThreads), (unsigned)cdiv(a.width, (int64_t)(VEC * U) << l));
    lookup_kernel<T, VEC, U><<<grid, kThreads, 0, s>>>(a, l);
    return cudaGetLastError();
}

// the widest vectors that the rows' starts and width allow
template <typename T>
cudaError_t lookup(const LookupArgs& a, cudaStream_t s) {
    constexpr int e = sizeof(T);
    const size_t all = reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.out) |
                       (a.table_stride * e) | (a.out_stride * e) | (a.width * e);
    if (all % 16 == 0) return lookup_by<T, 16 / e, 4>(a, s);
    if (all % 4 == 0) return lookup_by<T, 4 / e, 8>(a, s);
    if constexpr (e < 4) return lookup_by<T, 1, 16>(a, s);
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------- gradient

template <typename T, int VEC>
struct Grad {
    template <int B>
    struct Terms {
        Pack<T, VEC> x[B];
        __device__ __forceinline__ void load(const TermsOf& of, const uint2* entry, int64_t col) {
#pragma unroll
            for (int j = 0; j < B; ++j)
                x[j] = *reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(of.a.grad) +
                                                              (int64_t)entry[j].y * of.a.grad_stride + col);
        }
        __device__ __forceinline__ float at(int j, int e) const { return to_f32(x[j].v[e]); }
    };
};

// rows in 16-byte vectors of the gradient's type where all starts allow it
template <typename T, typename TO>
cudaError_t lookup_grad(const RowSumArgs& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    const size_t from = reinterpret_cast<uintptr_t>(a.grad) | (a.grad_stride * sizeof(T)) | (a.width * sizeof(T));
    const size_t to = reinterpret_cast<uintptr_t>(a.out[0]) | (a.out_stride * sizeof(TO));
    if (from % 16 == 0 && to % (kVec * sizeof(TO)) == 0) return sums_by<TO, kVec, 8, Grad<T, kVec>::template Terms>(a, s);
    return sums_by<TO, 1, 8, Grad<T, 1>::template Terms>(a, s);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, int type, cudaStream_t s) {
    if (a.index.n == 0) return cudaSuccess;
    if (type == MTTKRP_F32) return lookup<float>(a, s);
    if (type == MTTKRP_BF16) return lookup<__nv_bfloat16>(a, s);
    return lookup<__half>(a, s);
}

size_t lookup_grad_workspace_bytes(const IndexArgs& index, int64_t width) {
    return plan_sort(index, sizeof(uint2)).total() + part_bytes(index, width);
}

cudaError_t launch_lookup_grad(const RowSumArgs& a, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if (a.type == MTTKRP_F32) return lookup_grad<float, float>(a, s);
    if (a.type == MTTKRP_BF16)
        return a.out_type == MTTKRP_F32 ? lookup_grad<bf16, float>(a, s) : lookup_grad<bf16, bf16>(a, s);
    return a.out_type == MTTKRP_F32 ? lookup_grad<__half, float>(a, s) : lookup_grad<__half, __half>(a, s);
}

}  // namespace mk
