// Entries of a CP model at coordinates, and the gradient of every factor:
//   x_s = sum over r of prod over n of A_n(c_sn, r),
//   G_n(i, :) = sum over s with c_sn = i of g_s * prod over m != n of A_m(c_sm, :).
//
// Samples read rows of the factors at random, far more bytes in all than the factors
// have: what bounds both is how fast rows are gathered.  From the L2 cache a row of
// 128 bytes costs an SM about 4.5 cycles, from shared memory 1.  So where there are
// many samples, CTAs hold a slice of CS columns of all factors in shared memory; and
// where they fit, products of neighbouring modes' rows instead of the rows themselves,
// which makes the gathers fewer (Tables).  Small problems, and factors whose slices do
// not fit, gather from the caches.
#include "sums.cuh"

namespace mk {
namespace {

constexpr int kStageThreads = 1024;

// ---------------------------------------------------------------- tables in shared memory

struct StageArgs {
    IndexArgs index;
    const void* factor[MTTKRP_MAX_ORDER];
    int type;
    int64_t width;
};

// four elements from a row's column c on, zeros behind the last column
__device__ __forceinline__ float4 row4(const StageArgs& a, int mode, int64_t row, int64_t c) {
    float v[4];
    const int64_t at = row * a.width + c;
    if (a.type == MTTKRP_F32) {
        const float* p = static_cast<const float*>(a.factor[mode]) + at;
        if (c + 4 <= a.width && (reinterpret_cast<uintptr_t>(p) & 15) == 0)
            return *reinterpret_cast<const float4*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < a.width ? p[e] : 0.f;
    } else if (a.type == MTTKRP_BF16) {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.factor[mode]) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < a.width ? to_f32(p[e]) : 0.f;
    } else {
        const __half* p = static_cast<const __half*>(a.factor[mode]) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < a.width ? to_f32(p[e]) : 0.f;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float4 times(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

// Columns col0 .. col0 + CS of the tables: row r at tab[r * CS].  kAhead rows a thread
// are in flight.
template <int CS>
__device__ __forceinline__ void stage(const StageArgs& a, const Tables& t, int64_t col0, float* tab) {
    constexpr int kQuads = CS / 4, kAhead = 4;
    const int items = t.rows * kQuads;
    for (int i0 = threadIdx.x; i0 < items; i0 += kAhead * kStageThreads) {
        float4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kStageThreads;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i >= items) continue;
            const int r = i / kQuads;
            int g = 0;
            while (g + 1 < t.groups && t.group[g + 1].first <= r) ++g;
            uint32_t rest = (uint32_t)(r - t.group[g].first);
            for (int k = t.group[g].modes - 1; k >= 0; --k) {
                const int mode = t.group[g].mode[k];
                const uint32_t rows = (uint32_t)a.index.rows[mode];
                const uint32_t q = rest / rows;
                const float4 x = row4(a, mode, rest - q * rows, col0 + (i % kQuads) * 4);
                v[u] = k == t.group[g].modes - 1 ? x : times(v[u], x);
                rest = q;
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kStageThreads;
            if (i < items) *reinterpret_cast<float4*>(tab + (size_t)i * 4) = v[u];
        }
    }
}

// product of a sample's rows, as 16-bit numbers in lo and hi, at four columns
template <int CS>
__device__ __forceinline__ float4 product(const float* tab, int groups, uint32_t lo, uint32_t hi) {
    auto row = [&](uint32_t r) { return *reinterpret_cast<const float4*>(tab + r * CS); };
    float4 p = row(lo & 0xFFFFu);
    if (groups > 1) p = times(p, row(lo >> 16));
    if (groups > 2) p = times(p, row(hi & 0xFFFFu));
    if (groups > 3) p = times(p, row(hi >> 16));
    return p;
}

// ---------------------------------------------------------------- entries

// L lanes a sample, gathering from the caches.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) entries_kernel(const __grid_constant__ EntriesArgs a, int log2L) {
    const int L = 1 << log2L;
    const int lane = threadIdx.x & (L - 1);
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2L;
    const bool any = t < a.index.n;
    const bool inside = any && sort_key(a.index, t, 0) != kNone;
    float sum = 0.f;
    if (inside) {
        for (int64_t c = (int64_t)lane * VEC; c < a.width; c += (int64_t)VEC << log2L) {
            float v[VEC];
            for (int l = 0; l < a.index.d; ++l) {
                const Pack<T, VEC> x = *reinterpret_cast<const Pack<T, VEC>*>(
                    static_cast<const T*>(a.factor[l]) + index_at(a.index, t, l) * a.width + c);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = l == 0 ? to_f32(x.v[e]) : v[e] * to_f32(x.v[e]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += v[e];
        }
    }
    for (int o = L >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (any && lane == 0) a.out[t] = sum;
}

// A CTA has `share` consecutive samples and goes through the slices of CS columns.  A
// warp takes 32 samples at a time: each lane works out the table rows of one, then
// L = CS / 4 lanes form the products of L samples, one after the other, and add them
// up so that every lane ends with its own sample's sum.
template <int CS>
__global__ void __launch_bounds__(kStageThreads, 1) entries_staged_kernel(const __grid_constant__ EntriesArgs a,
                                                                          const __grid_constant__ StageArgs stage_args,
                                                                          const __grid_constant__ Tables tables,
                                                                          int64_t share) {
    extern __shared__ float4 stage_smem[];
    constexpr int L = CS / 4;
    float* tab = reinterpret_cast<float*>(stage_smem);
    const int lane = threadIdx.x & 31;
    const int64_t t0 = blockIdx.x * share;
    const int64_t t1 = t0 + share < a.index.n ? t0 + share : a.index.n;
    const float* mine = tab + (lane & (L - 1)) * 4;
    for (int64_t col0 = 0; col0 < a.width; col0 += CS) {
        stage<CS>(stage_args, tables, col0, tab);
        __syncthreads();
        for (int64_t base = t0 + (threadIdx.x & ~31); base < t1; base += kStageThreads) {
            const int64_t t = base + lane;
            const bool inside = t < t1 && sort_key(a.index, t, 0) != kNone;
            uint32_t lo = 0, hi = 0;
            if (inside) {
                uint32_t row[kMaxGroups] = {};
#pragma unroll
                for (int k = 0; k < kMaxGroups; ++k)
                    if (k < tables.groups) row[k] = table_row(a.index, tables.group[k], t);
                lo = row[0] | row[1] << 16;
                hi = row[2] | row[3] << 16;
            }
            float acc[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const float4 p = product<CS>(mine, tables.groups, __shfl_sync(0xFFFFFFFFu, lo, i, L),
                                             __shfl_sync(0xFFFFFFFFu, hi, i, L));
                acc[i] = (p.x + p.y) + (p.z + p.w);
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                const bool upper = (lane & o) != 0;
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const float send = upper ? acc[i] : acc[i + o];
                    acc[i] = (upper ? acc[i + o] : acc[i]) + __shfl_xor_sync(0xFFFFFFFFu, send, o);
                }
            }
            if (t < t1) a.out[t] = !inside ? 0.f : col0 == 0 ? acc[0] : a.out[t] + acc[0];
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- gradient

template <typename T, int VEC>
struct Model {
    template <int B>
    struct Terms {
        float v[B][VEC];
        __device__ __forceinline__ void load(const TermsOf& of, const uint2* entry, int64_t col) {
            const RowSumArgs& a = of.a;
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const float g = a.g[entry[j].y];
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] = g;
            }
            for (int l = 0; l < a.index.d; ++l) {
                if (l == of.m) continue;
                Pack<T, VEC> x[B];
#pragma unroll
                for (int j = 0; j < B; ++j)
                    x[j] = *reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(a.factor[l]) +
                                                                  index_at(a.index, entry[j].y, l) * a.width + col);
#pragma unroll
                for (int j = 0; j < B; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[j][e] *= to_f32(x[j].v[e]);
            }
        }
        __device__ __forceinline__ float at(int j, int e) const { return v[j][e]; }
    };
};

// terms of entries of 16 bytes from tables in shared memory
struct StagedOf {
    const float* tab;       // at the lane's columns
    int groups;
};

template <int CS, int VEC, int B>
struct StagedTerms {
    float v[B][VEC];
    __device__ __forceinline__ void load(const StagedOf& of, const uint4* entry, int64_t) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const float g = __uint_as_float(entry[j].y);
            if constexpr (VEC == 4) {
                float4 p = make_float4(1.f, 1.f, 1.f, 1.f);
                if (of.groups > 0) p = product<CS>(of.tab, of.groups, entry[j].z, entry[j].w);
                v[j][0] = g * p.x;
                v[j][1] = g * p.y;
                v[j][2] = g * p.z;
                v[j][3] = g * p.w;
            } else {
                float p = g;
                if (of.groups > 0) p *= of.tab[(entry[j].z & 0xFFFFu) * CS];
                if (of.groups > 1) p *= of.tab[(entry[j].z >> 16) * CS];
                if (of.groups > 2) p *= of.tab[(entry[j].w & 0xFFFFu) * CS];
                if (of.groups > 3) p *= of.tab[(entry[j].w >> 16) * CS];
                v[j][0] = p;
            }
        }
    }
    __device__ __forceinline__ float at(int j, int e) const { return v[j][e]; }
};

struct StagedArgs {
    SumArgs s;
    StageArgs stage;
    Tables tables[MTTKRP_MAX_ORDER];
};

// A CTA has a slice of CS columns (blockIdx.x) and s.tile sorted samples (blockIdx.y)
// of one mode (blockIdx.z).
template <int CS, int VEC>
__global__ void __launch_bounds__(kStageThreads, 1) staged_sum_kernel(const __grid_constant__ StagedArgs a) {
    extern __shared__ float4 stage_smem[];
    constexpr int L = CS / VEC, kLog2L = L == 32 ? 5 : L == 16 ? 4 : L == 8 ? 3 : L == 4 ? 2 : 1;
    static_assert(1 << kLog2L == L, "lanes of a sample");
    float* heads = reinterpret_cast<float*>(stage_smem);        // kStageThreads * VEC
    float* tab = heads + kStageThreads * VEC;
    const SumArgs& s = a.s;
    const int m = blockIdx.z;
    const int64_t n = s.a.index.n, col0 = (int64_t)blockIdx.x * CS;
    const uint4* sorted = reinterpret_cast<const uint4*>(s.sorted.entries) + m * n;
    const int64_t p0 = blockIdx.y * s.tile, p1 = p0 + s.tile < n ? p0 + s.tile : n;
    stage<CS>(a.stage, a.tables[m], col0, tab);
    // entries that take part come first: find the end in two steps of 1024 probes
    int64_t lo = p0, hi = p1;
    while (lo < hi) {
        const int64_t step = cdiv(hi - lo, kStageThreads);
        const int64_t p = lo + (int64_t)threadIdx.x * step;
        const int have = __syncthreads_count(p < hi && sorted[p].x != kNone);
        if (have == 0) hi = lo;
        else {
            const int64_t end = lo + have * step;
            lo += (have - 1) * step + 1;
            hi = end < hi ? end : hi;
        }
    }
    const int count = (int)(lo - p0);
    __syncthreads();
    if (count == 0) return;
    const uint4* list = sorted + p0;
    float* part = s.part + ((int64_t)m * s.tiles + blockIdx.y) * 2 * s.a.width;
    Around around;
    around.before = p0 > 0 && list[-1].x == list[0].x;
    around.after = p0 + count < n && list[count].x == list[count - 1].x;
    around.head = part;
    around.tail = part + s.a.width;
    const StagedOf of{tab + (threadIdx.x & (L - 1)) * VEC, a.tables[m].groups};
    sum_list<float, VEC, 4, StagedTerms<CS, VEC, 4>, kStageThreads>(
        s.a, m, of, [&](int p) { return __ldg(list + p); }, [](uint32_t v) { return v; }, count, kLog2L, col0, heads,
        around, [] { __syncthreads(); });
}

// ---------------------------------------------------------------- host

// What a step costs an SM, in cycles, by measurement on GB300: a gathered row slice of
// CS columns from shared memory (bank conflicts between rows of less than 128 bytes
// included) and from the L2 cache (32 columns of fp32), the rest of a sample and slice,
// and the start of a slice's tables with the load of a row.
constexpr double kGather32 = 1.0, kGather16 = 0.75, kGather8 = 0.53;
constexpr double kGatherCache = 4.5;
constexpr double kSample = 1.3;
constexpr double kStageStart = 3000.0, kStageRow = 3.0;

double gather_cost(int cs) { return cs == 32 ? kGather32 : cs == 16 ? kGather16 : kGather8; }

// The tables with the least work for `samples` samples an SM among the ways to split
// the d modes but `skip` into consecutive groups; returns that work (a negative number
// where no way fits max_rows rows and kMaxGroups groups).
double plan_tables(const IndexArgs& x, int skip, int cs, int64_t max_rows, double samples, Tables& best) {
    int mode[MTTKRP_MAX_ORDER], modes = 0;
    for (int m = 0; m < x.d; ++m)
        if (m != skip) mode[modes++] = m;
    double least = -1.0;
    for (int cuts = 0; cuts < (modes > 0 ? 1 << (modes - 1) : 1); ++cuts) {
        Tables t;
        t.groups = 0;
        int64_t rows = 0;
        double work = kStageStart;
        bool fits = true;
        for (int k = 0; k < modes && fits;) {
            if (t.groups == kMaxGroups) {
                fits = false;
                break;
            }
            Tables::Group& g = t.group[t.groups++];
            g.first = (int)rows;
            g.modes = 0;
            int64_t size = 1;
            do {
                size *= x.rows[mode[k]];
                g.mode[g.modes++] = mode[k++];
                fits = fits && size <= max_rows;
            } while (fits && k < modes && (cuts >> (k - 1) & 1) == 0);
            rows += size;
            work += (double)size * g.modes * kStageRow * cs / 32;
        }
        if (!fits || rows > max_rows) continue;
        t.rows = (int)rows;
        work += samples * (t.groups * gather_cost(cs) + kSample);
        if (least < 0.0 || work < least) {
            least = work;
            best = t;
        }
    }
    return least;
}

int64_t table_rows(size_t other_smem, int cs) {
    const int64_t rows = (int64_t)(kMaxSmem - other_smem) / (cs * 4);
    return rows < 65536 ? rows : 65535;
}

template <typename T>
bool wide_rows(const void* p, int64_t width) {
    return ((reinterpret_cast<uintptr_t>(p) | (width * sizeof(T))) & 15) == 0;
}

template <typename T>
cudaError_t entries_cached(const EntriesArgs& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    bool w = true;
    for (int m = 0; m < a.index.d; ++m) w = w && wide_rows<T>(a.factor[m], a.width);
    int l = 0;
    while (l < 5 && ((int64_t)(w ? kVec : 1) << l) < a.width) ++l;
    const unsigned blocks = (unsigned)cdiv(a.index.n << l, kThreads);
    if (w) entries_kernel<T, kVec><<<blocks, kThreads, 0, s>>>(a, l);
    else entries_kernel<T, 1><<<blocks, kThreads, 0, s>>>(a, l);
    return cudaGetLastError();
}

StageArgs stage_args(const IndexArgs& index, const void* const* factor, int type, int64_t width) {
    StageArgs a;
    a.index = index;
    for (int m = 0; m < index.d; ++m) a.factor[m] = factor[m];
    a.type = type;
    a.width = width;
    return a;
}

template <int CS>
cudaError_t entries_staged(const EntriesArgs& a, const Tables& t, int64_t share, cudaStream_t s) {
    cudaError_t e = allow_smem<entries_staged_kernel<CS>>();
    if (e != cudaSuccess) return e;
    entries_staged_kernel<CS><<<(unsigned)cdiv(a.index.n, share), kStageThreads, sizeof(float) * t.rows * CS, s>>>(
        a, stage_args(a.index, a.factor, a.type, a.width), t, share);
    return cudaGetLastError();
}

template <typename T>
cudaError_t grad_cached(const RowSumArgs& a, cudaStream_t s) {
    bool w = a.width % 4 == 0;
    for (int m = 0; m < a.index.d; ++m)
        w = w && (reinterpret_cast<uintptr_t>(a.factor[m]) % (4 * sizeof(T))) == 0 &&
            (reinterpret_cast<uintptr_t>(a.out[m]) % (4 * sizeof(float))) == 0;
    if (w) return sums_by<float, 4, 4, Model<T, 4>::template Terms>(a, s);
    return sums_by<float, 1, 4, Model<T, 1>::template Terms>(a, s);
}

template <int CS, int VEC>
cudaError_t grad_staged(StagedArgs& a, const SortPlan& p, cudaStream_t st) {
    const RowSumArgs& r = a.s.a;
    int rows = 0;
    for (int m = 0; m < r.index.d; ++m) rows = a.tables[m].rows > rows ? a.tables[m].rows : rows;
    cudaError_t e = allow_smem<staged_sum_kernel<CS, VEC>>();
    if (e == cudaSuccess) e = sort_tokens(r.index, p, r.ws, a.tables, r.g, a.s.sorted, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)cdiv(r.width, CS), (unsigned)a.s.tiles, r.index.d);
    const size_t smem = sizeof(float) * (kStageThreads * VEC + (size_t)rows * CS);
    staged_sum_kernel<CS, VEC><<<grid, kStageThreads, smem, st>>>(a);
    return finish<float, VEC>(a.s, st);
}

}  // namespace

cudaError_t launch_entries(const EntriesArgs& a, cudaStream_t s) {
    const int64_t n = a.index.n;
    if (n == 0) return cudaSuccess;
    const int64_t share = cdiv(cdiv(n, kSms), 32) * 32;
    double least = kGatherCache * a.index.d * cdiv(a.width, 32) * (double)n / kSms;
    int cs = 0;
    Tables tables;
    for (int c = 32; c >= 8; c /= 2) {
        Tables t;
        const double slice = plan_tables(a.index, -1, c, table_rows(0, c), (double)share, t);
        const double work = slice * cdiv(a.width, c);
        if (slice >= 0.0 && work < least) {
            least = work;
            tables = t;
            cs = c;
        }
    }
    if (cs == 32) return entries_staged<32>(a, tables, share, s);
    if (cs == 16) return entries_staged<16>(a, tables, share, s);
    if (cs == 8) return entries_staged<8>(a, tables, share, s);
    if (a.type == MTTKRP_F32) return entries_cached<float>(a, s);
    if (a.type == MTTKRP_BF16) return entries_cached<__nv_bfloat16>(a, s);
    return entries_cached<__half>(a, s);
}

// for the larger entries that the sums from shared memory sort
size_t entries_grad_workspace_bytes(const IndexArgs& index, int64_t width) {
    return plan_sort(index, sizeof(uint4)).total() + part_bytes(index, width);
}

cudaError_t launch_entries_grad(const RowSumArgs& a, cudaStream_t s) {
    const int64_t n = a.index.n;
    const int d = a.index.d;
    bool quads = a.width % 4 == 0;
    for (int m = 0; m < d; ++m) quads = quads && reinterpret_cast<uintptr_t>(a.out[m]) % 16 == 0;
    const int vec = quads ? 4 : 1;
    double least = kGatherCache * d * (d - 1) * cdiv(a.width, 32) * (double)n / kSms;
    int cs = 0;
    StagedArgs st;
    for (int c = 32; c >= 8 && n > kOwnTokens; c /= 2) {
        const int64_t combos = cdiv(a.width, c) * d;
        int64_t tiles = combos < kSms ? kSms / combos : 1;
        tiles = tiles < cdiv(n, kTile) ? tiles : cdiv(n, kTile);
        const int64_t waves = cdiv(combos * tiles, kSms);
        double work = 0.0;
        Tables t[MTTKRP_MAX_ORDER];
        for (int m = 0; m < d && work >= 0.0; ++m) {
            const double slice = plan_tables(a.index, m, c, table_rows(sizeof(float) * kStageThreads * vec, c),
                                             (double)n / tiles, t[m]);
            work = slice < 0.0 ? -1.0 : (slice > work ? slice : work);
        }
        if (work >= 0.0 && work * waves < least) {
            least = work * waves;
            cs = c;
            for (int m = 0; m < d; ++m) st.tables[m] = t[m];
            st.s.tile = cdiv(n, tiles);
            st.s.tiles = cdiv(n, st.s.tile);
        }
    }
    if (cs != 0) {
        const SortPlan p = plan_sort(a.index, sizeof(uint4));
        st.s.a = a;
        st.s.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + p.total());
        st.stage = stage_args(a.index, a.factor, a.type, a.width);
        if (cs == 32) return quads ? grad_staged<32, 4>(st, p, s) : grad_staged<32, 1>(st, p, s);
        if (cs == 16) return quads ? grad_staged<16, 4>(st, p, s) : grad_staged<16, 1>(st, p, s);
        return quads ? grad_staged<8, 4>(st, p, s) : grad_staged<8, 1>(st, p, s);
    }
    if (a.type == MTTKRP_F32) return grad_cached<float>(a, s);
    if (a.type == MTTKRP_BF16) return grad_cached<__nv_bfloat16>(a, s);
    return grad_cached<__half>(a, s);
}

}  // namespace mk
