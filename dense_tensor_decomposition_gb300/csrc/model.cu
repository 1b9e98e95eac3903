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
#include <type_traits>

#include "sums.cuh"

namespace mk {
namespace {

constexpr int kStageThreads = 1024;

// ---------------------------------------------------------------- tables in shared memory

struct StageArgs {
    IndexArgs index;
    const void* factor[MTTKRP_MAX_ORDER];
    uint32_t inverse[MTTKRP_MAX_ORDER];     // of a mode's rows, see stage()
    int type;
    bool quads;             // fp32, and every four columns stand at a multiple of 16 bytes
    int64_t width;
};

// four elements from a row's column c on, zeros behind the last column
__device__ __forceinline__ float4 row4(const StageArgs& a, int mode, uint32_t row, int64_t c) {
    const int64_t at = (int64_t)row * a.width + c;
    if (a.quads)
        return c < a.width ? *reinterpret_cast<const float4*>(static_cast<const float*>(a.factor[mode]) + at)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = 0.f;
        if (c + e >= a.width) continue;
        if (a.type == MTTKRP_F32) v[e] = static_cast<const float*>(a.factor[mode])[at + e];
        else if (a.type == MTTKRP_BF16) v[e] = to_f32(static_cast<const __nv_bfloat16*>(a.factor[mode])[at + e]);
        else v[e] = to_f32(static_cast<const __half*>(a.factor[mode])[at + e]);
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float4 times(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

// Columns col0 .. col0 + CS of the tables: row r at tab[r * CS].  A group of CS / 4
// lanes takes a row, kAhead rows in turn.
template <int CS>
__device__ __forceinline__ void stage(const StageArgs& a, const Tables& t, int64_t col0, float* tab) {
    constexpr int kQuads = CS / 4, kGroups = kStageThreads / kQuads, kAhead = 4;
    const int64_t c = col0 + (threadIdx.x % kQuads) * 4;
    float* to = tab + (threadIdx.x % kQuads) * 4;
    for (int g = 0; g < t.groups; ++g) {
        const Tables::Group& group = t.group[g];
        const uint32_t rows = (uint32_t)((g + 1 < t.groups ? t.group[g + 1].first : t.rows) - group.first);
        for (uint32_t r0 = threadIdx.x / kQuads; r0 < rows; r0 += kAhead * kGroups) {
            float4 v[kAhead];
            uint32_t rest[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                rest[u] = min(r0 + u * kGroups, rows - 1);
                v[u] = make_float4(1.f, 1.f, 1.f, 1.f);
            }
            for (int k = group.modes - 1; k >= 0; --k) {
                const int mode = group.mode[k];
                const uint32_t size = (uint32_t)a.index.rows[mode], inverse = a.inverse[mode];
                float4 x[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    // rest / size for both below 2^16: inverse is 2^32 / size rounded up (0 for size 1)
                    const uint32_t q = k == 0 ? 0 : inverse == 0 ? rest[u] : __umulhi(rest[u], inverse);
                    x[u] = row4(a, mode, rest[u] - q * size, c);
                    rest[u] = q;
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) v[u] = times(v[u], x[u]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t r = r0 + u * kGroups;
                if (r < rows) *reinterpret_cast<float4*>(to + (size_t)(group.first + r) * CS) = v[u];
            }
        }
    }
}

// a sample's rows in G tables, as 16-bit numbers
template <int G>
struct alignas(G > kFewGroups ? 16 : 8) Rows {
    static constexpr int kWords = G > kFewGroups ? kMaxGroups / 2 : kFewGroups / 2;
    uint32_t w[kWords];
    __device__ __forceinline__ uint32_t row(int k) const { return k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xFFFFu; }
};

// the product of the rows at the four columns from tab on
template <int CS, int G>
__device__ __forceinline__ Pack<float, 4> product(const float* tab, const Rows<G>& r) {
    using P = Pack<float, 4>;
    P p = *reinterpret_cast<const P*>(tab + r.row(0) * CS);
#pragma unroll
    for (int k = 1; k < G; ++k) {
        const P x = *reinterpret_cast<const P*>(tab + r.row(k) * CS);
#pragma unroll
        for (int e = 0; e < 4; ++e) p.v[e] *= x.v[e];
    }
    return p;
}

// ---------------------------------------------------------------- entries

// L lanes a sample (up to a CTA's where samples are few and the rank is large), gathering
// from the caches.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) entries_kernel(const __grid_constant__ EntriesArgs a, int log2L) {
    after_previous();
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
    for (int o = L < 32 ? L >> 1 : 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (L > 32) {
        __shared__ float warps[kThreads / 32];
        if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (lane == 0)
            for (int w = 1; w < L >> 5; ++w) sum += warps[(threadIdx.x >> 5) + w];
    }
    if (any && lane == 0) a.out[t] = sum;
}

// A CTA has `share` consecutive samples and goes through the slices of CS columns.  The
// samples' table rows stand behind the tables, worked out once.  A warp takes 32 samples
// at a time: L = CS / 4 lanes form the products of L samples, one after the other, and
// add them up so that every lane ends with its own sample's sum.
// bytes of shared memory for 32 samples
constexpr int sample_bytes(int groups) { return 32 * (groups > kFewGroups ? sizeof(Rows<kMaxGroups>) : sizeof(Rows<1>)) + 4; }

template <int CS, int G>
__global__ void __launch_bounds__(kStageThreads, 1) entries_staged_kernel(const __grid_constant__ EntriesArgs a,
                                                                          const __grid_constant__ StageArgs stage_args,
                                                                          const __grid_constant__ Tables tables,
                                                                          int share) {
    extern __shared__ float4 stage_smem[];
    constexpr int L = CS / 4;
    float* tab = reinterpret_cast<float*>(stage_smem);
    Rows<G>* rows = reinterpret_cast<Rows<G>*>(tab + (size_t)tables.rows * CS);
    uint32_t* parts = reinterpret_cast<uint32_t*>(rows + share);                // a bit a sample: it takes part
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * share;
    const int count = (int)(t0 + share < a.index.n ? share : a.index.n - t0);
    // samples that take no part, and those behind the last one of a warp's 32, read row 0
    for (int i = threadIdx.x; i < (count + 31) / 32 * 32; i += kStageThreads) {
        Rows<G> r = {};
        const bool inside = i < count && sort_key(a.index, t0 + i, 0) != kNone;
        if (inside) {
#pragma unroll
            for (int k = 0; k < G; ++k) r.w[k / 2] |= table_row(a.index, tables.group[k], t0 + i) << (k & 1) * 16;
        }
        rows[i] = r;
        const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, inside);
        if (lane == 0) parts[i / 32] = ballot;
    }
    const float* mine = tab + (lane & (L - 1)) * 4;
    for (int64_t col0 = 0; col0 < a.width; col0 += CS) {
        stage<CS>(stage_args, tables, col0, tab);
        __syncthreads();
        for (int base = threadIdx.x & ~31; base < count; base += kStageThreads) {
            const int i = base + lane;
            float acc[L];
#pragma unroll
            for (int k = 0; k < L; ++k) {
                const Pack<float, 4> p = product<CS, G>(mine, rows[base + (lane & ~(L - 1)) + k]);
                acc[k] = (p.v[0] + p.v[1]) + (p.v[2] + p.v[3]);
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                const bool upper = (lane & o) != 0;
#pragma unroll
                for (int k = 0; k < o; ++k) {
                    const float send = upper ? acc[k] : acc[k + o];
                    acc[k] = (upper ? acc[k + o] : acc[k]) + __shfl_xor_sync(0xFFFFFFFFu, send, o);
                }
            }
            if (i < count) {
                float* x = a.out + t0 + i;
                *x = (parts[i / 32] >> lane & 1u) == 0 ? 0.f : col0 == 0 ? acc[0] : *x + acc[0];
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- gradient

// products of factor rows from the caches
template <typename T, int VEC>
struct Model {
    template <typename List>
    struct Terms {
        static constexpr int kB = 4;
        static constexpr bool kAllLanes = false;
        const TermsOf& of;
        const List& list;
        const int p1;
        const int64_t col;
        uint32_t keys[kB];
        float v[kB][VEC];
        __device__ __forceinline__ Terms(const TermsOf& of, const List& list, int, int p1, int64_t col)
            : of(of), list(list), p1(p1), col(col) {}
        __device__ __forceinline__ void load(int p) {
            const RowSumArgs& a = of.a;
            uint32_t tok[kB];
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                const uint2 entry = list(p + j < p1 ? p + j : p);
                keys[j] = entry.x;
                tok[j] = entry.y;
                const float g = a.g[tok[j]];
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] = g;
            }
            for (int l = 0; l < a.index.d; ++l) {
                if (l == of.m) continue;
                using P = Pack<T, VEC>;
                using Raw = typename Bits<sizeof(P)>::type;
                Raw x[kB];
#pragma unroll
                for (int j = 0; j < kB; ++j)
                    x[j] = *reinterpret_cast<const Raw*>(static_cast<const T*>(a.factor[l]) +
                                                         index_at(a.index, tok[j], l) * a.width + col);
#pragma unroll
                for (int j = 0; j < kB; ++j) {
                    const P p = as_pack<P>(x[j]);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[j][e] *= to_f32(p.v[e]);
                }
            }
        }
        __device__ __forceinline__ uint32_t key(int j) const { return keys[j]; }
        __device__ __forceinline__ void add(int j, float* acc) const {
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += v[j][e];
        }
    };
};

// Products of table rows in shared memory, of entries of 16 bytes.  The L lanes of a
// sample hold L entries, one each, which go round by shuffles (reading every entry in
// every lane would take as many shared-memory cycles as half a table row); the next L
// are on their way meanwhile.
struct StagedOf {
    const float* tab;       // at the lane's columns
};

template <int G>
struct Entry {
    uint32_t x;                 // the row
    float g;
    Rows<G> rows;
};

// Entry p of a list of entries of 16 or 32 bytes.  By plain loads: the sort before this
// launch writes the list, and loads by the read-only path need not stay behind
// after_previous().
template <int G>
__device__ __forceinline__ Entry<G> entry_at(const char* list, int64_t p) {
    constexpr int kBytes = G > kFewGroups ? 32 : 16;
    const uint4 a = *reinterpret_cast<const uint4*>(list + p * kBytes);
    Entry<G> e;
    e.x = a.x;
    e.g = __uint_as_float(a.y);
    e.rows.w[0] = a.z;
    e.rows.w[1] = a.w;
    if constexpr (G > kFewGroups) {
        const uint2 b = *reinterpret_cast<const uint2*>(list + p * kBytes + 16);
        e.rows.w[2] = b.x;
        e.rows.w[3] = b.y;
    }
    return e;
}

template <int CS, int G>
struct Staged {
    template <typename List>
    struct Terms {
        static constexpr int L = CS / 4, kB = L < 4 ? L : 4;
        static constexpr bool kAllLanes = true;
        const StagedOf& of;
        const List& list;
        const int p0, p1;
        const uint32_t lanes;       // of the group
        int at;                     // which of the held entries is token p of load(p)
        Entry<G> held, next;
        __device__ __forceinline__ Terms(const StagedOf& of, const List& list, int p0, int p1, int64_t)
            : of(of), list(list), p0(p0), p1(p1),
              lanes((0xFFFFFFFFu >> (32 - L)) << (threadIdx.x & 31 & ~(L - 1))), at(0) {
            fetch(p0);
        }
        __device__ __forceinline__ void fetch(int p) {
            const int own = p + (threadIdx.x & (L - 1));
            next = list(own < p1 ? own : p1 - 1);
        }
        __device__ __forceinline__ void load(int p) {
            at = (p - p0) & (L - 1);
            if (at == 0) {
                held = next;
                fetch(p + L);
            }
        }
        __device__ __forceinline__ uint32_t key(int j) const { return __shfl_sync(lanes, held.x, at + j, L); }
        __device__ __forceinline__ void add(int j, float* acc) const {
            const float g = __shfl_sync(lanes, held.g, at + j, L);
            Rows<G> r;
#pragma unroll
            for (int w = 0; w < (G + 1) / 2; ++w) r.w[w] = __shfl_sync(lanes, held.rows.w[w], at + j, L);
            const Pack<float, 4> p = product<CS, G>(of.tab, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(g, p.v[e], acc[e]);
        }
    };
};

struct StagedArgs {
    SumArgs s;
    StageArgs stage;
    Tables tables[MTTKRP_MAX_ORDER];
};

// A CTA (blockIdx.x) has a slice of CS columns and s.tile sorted samples of one mode
// (blockIdx.y); those behind the slices' and tiles' write zeros, 32 rows a warp.
template <int CS, bool kRagged, bool kMany>
__global__ void __launch_bounds__(kStageThreads, 1) staged_sum_kernel(const __grid_constant__ StagedArgs a) {
    extern __shared__ float4 stage_smem[];
    constexpr int L = CS / 4, kLog2L = L == 8 ? 3 : L == 4 ? 2 : 1;
    static_assert(1 << kLog2L == L, "lanes of a sample");
    float* heads = reinterpret_cast<float*>(stage_smem);        // kStageThreads * 4
    float* tab = heads + kStageThreads * 4;
    const SumArgs& s = a.s;
    const int m = blockIdx.y;
    const int64_t n = s.a.index.n;
    const uint32_t tile = blockIdx.x % (uint32_t)s.tiles, slice = blockIdx.x / (uint32_t)s.tiles;
    const int64_t col0 = (int64_t)slice * CS;
    // the factors were there before the sort, this launch's previous one, began
    if (col0 < s.a.width) stage<CS>(a.stage, a.tables[m], col0, tab);
    after_previous();
    if (col0 >= s.a.width) {
        const int64_t warp = (blockIdx.x - cdiv(s.a.width, CS) * s.tiles) * (kStageThreads / 32) + (threadIdx.x >> 5);
        zero_unsorted_rows<float, kRagged ? 1 : 4>(s.a, m, warp * 32, [&](int64_t p) { return key_at(s, m, p); });
        return;
    }
    const int64_t p0 = tile * s.tile, p1 = p0 + s.tile < n ? p0 + s.tile : n;
    // entries that take part come first: find the end in two steps of 1024 probes
    int64_t lo = p0, hi = p1;
    while (lo < hi) {
        const int64_t step = cdiv(hi - lo, kStageThreads);
        const int64_t p = lo + (int64_t)threadIdx.x * step;
        const int have = __syncthreads_count(p < hi && key_at(s, m, p) != kNone);
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
    const char* list = s.sorted.entries + (m * n + p0) * s.sorted.bytes;
    float* part = s.part + ((int64_t)m * s.tiles + tile) * 2 * s.a.width;
    Around around;
    around.before = p0 > 0 && key_at(s, m, p0 - 1) == key_at(s, m, p0);
    around.after = p0 + count < n && key_at(s, m, p0 + count) == key_at(s, m, p0 + count - 1);
    around.head = part;
    around.tail = part + s.a.width;
    const StagedOf of{tab + (threadIdx.x & (L - 1)) * 4};
    auto sum = [&](auto g) {
        constexpr int G = decltype(g)::value;
        sum_list<float, 4, Staged<CS, G>::template Terms, kStageThreads, kRagged>(
            s.a, m, of, [&](int p) { return entry_at<G>(list, p); }, [](uint32_t v) { return v; }, count, kLog2L, col0,
            heads, around, [] { __syncthreads(); });
    };
    const int groups = a.tables[m].groups;
    if constexpr (kMany) {
        if (groups == 7) sum(std::integral_constant<int, 7>());
        else if (groups == 6) sum(std::integral_constant<int, 6>());
        else sum(std::integral_constant<int, 5>());
    } else {
        if (groups == 1) sum(std::integral_constant<int, 1>());
        else if (groups == 2) sum(std::integral_constant<int, 2>());
        else if (groups == 3) sum(std::integral_constant<int, 3>());
        else sum(std::integral_constant<int, 4>());
    }
}

// ---------------------------------------------------------------- host

// What a step costs an SM, in cycles, by measurement on GB300: a gathered row slice of
// CS columns from shared memory (bank conflicts between rows of less than 128 bytes
// included) and from the L2 cache (32 columns of fp32), the rest of a sample and slice,
// and the start of a slice's tables with the load of a row.  Factors of 16 bits, and in
// launch_entries() ranks that are read one column a load, are planned with the same
// figures (tables hold fp32 whatever the factors' type).
constexpr double kGather32 = 1.0, kGather16 = 0.75, kGather8 = 0.53;
constexpr double kGatherCache = 4.5;
constexpr double kSample = 1.3;
constexpr double kStageStart = 3000.0, kStageRow = 3.0;
constexpr double kSortAndJoin = 40000.0;        // what else the sums from tables take, where few samples go without

double gather_cost(int cs) { return cs == 32 ? kGather32 : cs == 16 ? kGather16 : kGather8; }

// An SM's work on tables: cycles to build them, and for a sample.
struct Work {
    double build = -1.0, sample = 0.0;      // build < 0: there are no such tables
    double of(double samples) const { return build + samples * sample; }
};

// The tables with the least work for `samples` samples an SM among the ways to split
// the d modes but `skip` into at most max_groups consecutive groups of max_rows rows in all.
Work plan_tables(const IndexArgs& x, int skip, int cs, int64_t max_rows, int max_groups, double samples,
                 Tables& best) {
    int mode[MTTKRP_MAX_ORDER], modes = 0;
    for (int m = 0; m < x.d; ++m)
        if (m != skip) mode[modes++] = m;
    Work least;
    for (int cuts = 0; cuts < (modes > 0 ? 1 << (modes - 1) : 1); ++cuts) {
        Tables t;
        t.groups = 0;
        int64_t rows = 0;
        Work work;
        work.build = kStageStart;
        bool fits = true;
        for (int k = 0; k < modes && fits;) {
            if (t.groups == max_groups) {
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
            work.build += (double)size * g.modes * kStageRow * cs / 32;
        }
        if (!fits || rows > max_rows) continue;
        t.rows = (int)rows;
        work.sample = t.groups * gather_cost(cs) + kSample;
        if (least.build < 0.0 || work.of(samples) < least.of(samples)) {
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
    while (((int64_t)(w ? kVec : 1) << l) < a.width && (l < 5 || (l < 8 && a.index.n << l < kSms * 1024))) ++l;
    const unsigned blocks = (unsigned)cdiv(a.index.n << l, kThreads);
    return launch_early(w ? entries_kernel<T, kVec> : entries_kernel<T, 1>, blocks, kThreads, 0, s, a, l);
}

StageArgs stage_args(const IndexArgs& index, const void* const* factor, int type, int64_t width) {
    StageArgs a;
    a.index = index;
    for (int m = 0; m < index.d; ++m) a.factor[m] = factor[m];
    a.type = type;
    a.quads = type == MTTKRP_F32 && width % 4 == 0;
    for (int m = 0; m < index.d; ++m) {
        a.quads = a.quads && reinterpret_cast<uintptr_t>(factor[m]) % 16 == 0;
        a.inverse[m] = (uint32_t)((((uint64_t)1 << 32) + index.rows[m] - 1) / index.rows[m]);
    }
    a.width = width;
    return a;
}

template <int CS, int G>
cudaError_t entries_staged(const EntriesArgs& a, const Tables& t, int64_t share, cudaStream_t s) {
    constexpr auto kernel = entries_staged_kernel<CS, G>;
    cudaError_t e = allow_smem<kernel>();
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(float) * t.rows * CS + sample_bytes(G) * share / 32;
    return launch_early(kernel, (unsigned)cdiv(a.index.n, share), kStageThreads, smem, s, a,
                        stage_args(a.index, a.factor, a.type, a.width), t, (int)share);
}

template <int CS>
cudaError_t entries_staged(const EntriesArgs& a, const Tables& t, int64_t share, cudaStream_t s) {
    switch (t.groups) {
        case 1: return entries_staged<CS, 1>(a, t, share, s);
        case 2: return entries_staged<CS, 2>(a, t, share, s);
        case 3: return entries_staged<CS, 3>(a, t, share, s);
        case 4: return entries_staged<CS, 4>(a, t, share, s);
        case 5: return entries_staged<CS, 5>(a, t, share, s);
        case 6: return entries_staged<CS, 6>(a, t, share, s);
        case 7: return entries_staged<CS, 7>(a, t, share, s);
        default: return entries_staged<CS, 8>(a, t, share, s);
    }
}

template <typename T>
cudaError_t grad_cached(const RowSumArgs& a, cudaStream_t s) {
    bool w = a.width % 4 == 0;
    for (int m = 0; m < a.index.d; ++m)
        w = w && (reinterpret_cast<uintptr_t>(a.factor[m]) % (4 * sizeof(T))) == 0 &&
            (reinterpret_cast<uintptr_t>(a.out[m]) % (4 * sizeof(float))) == 0;
    if (w) return sums_by<float, 4, Model<T, 4>::template Terms, 0, Model<T, 4>::template Terms, 0>(a, s);
    return sums_by<float, 1, Model<T, 1>::template Terms, 0, Model<T, 1>::template Terms, 0>(a, s);
}

template <int CS, bool kRagged, bool kMany>
cudaError_t grad_staged(StagedArgs& a, cudaStream_t st) {
    const RowSumArgs& r = a.s.a;
    const SortPlan p = plan_sort(r.index, kMany ? 32 : 16, sort_sms());
    a.s.part = reinterpret_cast<float*>(static_cast<char*>(r.ws) + p.total());
    int rows = 0;
    for (int m = 0; m < r.index.d; ++m) rows = a.tables[m].rows > rows ? a.tables[m].rows : rows;
    constexpr auto kernel = staged_sum_kernel<CS, kRagged, kMany>;
    cudaError_t e = allow_smem<kernel>();
    if (e == cudaSuccess) e = sort_tokens(r.index, p, r.ws, a.tables, r.g, a.s.sorted, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(cdiv(r.width, CS) * a.s.tiles + cdiv(most_rows(r.index), kStageThreads)), r.index.d);
    const size_t smem = sizeof(float) * (kStageThreads * 4 + (size_t)rows * CS);
    e = launch_early(kernel, grid, kStageThreads, smem, st, a);
    if (e != cudaSuccess) return e;
    return join<float, kRagged ? 1 : 4>(a.s, st);
}

// ragged: results are not written in vectors of four columns
template <int CS>
cudaError_t grad_staged(StagedArgs& a, bool ragged, cudaStream_t st) {
    bool many = false;
    for (int m = 0; m < a.s.a.index.d; ++m) many = many || a.tables[m].groups > kFewGroups;
    if (!many) return ragged ? grad_staged<CS, true, false>(a, st) : grad_staged<CS, false, false>(a, st);
    // every mode gets more than kFewGroups groups: those that lack some, tables of a row of ones
    for (int m = 0; m < a.s.a.index.d; ++m) {
        Tables& t = a.tables[m];
        while (t.groups <= kFewGroups) {
            t.group[t.groups].modes = 0;
            t.group[t.groups++].first = t.rows++;
        }
    }
    return ragged ? grad_staged<CS, true, true>(a, st) : grad_staged<CS, false, true>(a, st);
}

}  // namespace

cudaError_t launch_entries(const EntriesArgs& a, cudaStream_t s) {
    const int64_t n = a.index.n;
    if (n == 0) return cudaSuccess;
    double least = kGatherCache * a.index.d * cdiv(a.width, 32) * (double)n / kSms;
    int cs = 0;
    int64_t share = 0;
    Tables tables;
    // tables cost at least their start
    const bool small = least < kStageStart * cdiv(a.width, 32);
    for (int c = 32; c >= 8 && !small; c /= 2) {
        for (int groups : {kFewGroups, kMaxGroups}) {
            // as few rounds of CTAs over the SMs as leave two thirds of the shared memory to the tables
            const int64_t most = kMaxSmem / 3 / sample_bytes(groups) * 32;
            const int64_t rounds = cdiv(n, kSms * most);
            const int64_t part = cdiv(cdiv(n, kSms * rounds), 32) * 32;
            Tables t;
            const Work slice = plan_tables(a.index, -1, c, table_rows(sample_bytes(groups) * part / 32, c), groups,
                                           (double)part, t);
            const double work = slice.of((double)part) * cdiv(a.width, c) * rounds;
            if (slice.build >= 0.0 && work < least) {
                least = work;
                tables = t;
                share = part;
                cs = c;
            }
        }
    }
    if (cs == 32) return entries_staged<32>(a, tables, share, s);
    if (cs == 16) return entries_staged<16>(a, tables, share, s);
    if (cs == 8) return entries_staged<8>(a, tables, share, s);
    if (a.type == MTTKRP_F32) return entries_cached<float>(a, s);
    if (a.type == MTTKRP_BF16) return entries_cached<__nv_bfloat16>(a, s);
    return entries_cached<__half>(a, s);
}

namespace {

// cycles an SM for the sums with rows from the caches; single columns a lane take about
// as long for a load as quads, and few tokens have few warps to wait for them
double cached_grad_work(const IndexArgs& x, int64_t width, int vec) {
    const double slow = vec == 4 ? 1.0 : x.n <= kOwnTokens ? 4.0 : 2.0;
    return slow * kGatherCache * x.d * (x.d - 1) * cdiv(width, 32) * (double)x.n / kSms;
}

// more than the fixed part of sums from tables
bool tables_may_pay(const IndexArgs& x, int64_t width, int vec) {
    return cached_grad_work(x, width, vec) > kStageStart + (x.n <= kOwnTokens ? kSortAndJoin : 0.0);
}

}  // namespace

// for the largest entries that the sums from shared memory can sort
size_t entries_grad_workspace_bytes(const IndexArgs& index, int64_t width) {
    if (always_owned(index, width) && !tables_may_pay(index, width, 1)) return 0;
    return plan_sort(index, index.d - 1 > kFewGroups ? 32 : 16, kSms).total() + part_bytes(index, width);
}

cudaError_t launch_entries_grad(const RowSumArgs& a, cudaStream_t s) {
    const int64_t n = a.index.n;
    const int d = a.index.d;
    bool quads = a.width % 4 == 0;
    for (int m = 0; m < d; ++m) quads = quads && reinterpret_cast<uintptr_t>(a.out[m]) % 16 == 0;
    const int vec = quads ? 4 : 1;
    double least = cached_grad_work(a.index, a.width, vec);
    int cs = 0;
    StagedArgs st;
    for (int c = 32; c >= 8 && tables_may_pay(a.index, a.width, vec); c /= 2) {
        const int64_t combos = cdiv(a.width, c) * d;
        Tables t[MTTKRP_MAX_ORDER];
        Work work[MTTKRP_MAX_ORDER];
        bool fits = true;
        for (int m = 0; m < d && fits; ++m) {
            work[m] = plan_tables(a.index, m, c, table_rows(sizeof(float) * kStageThreads * 4, c) - kMaxGroups,
                                  kMaxGroups, (double)n * combos / kSms, t[m]);
            fits = work[m].build >= 0.0;
        }
        // in how many tiles: the last round of CTAs over the SMs should not leave many without
        const int64_t most = cdiv(n, tile_tokens(n)) < kSms ? cdiv(n, tile_tokens(n)) : kSms;     // part_bytes()
        for (int64_t tiles = 1; tiles <= most && fits; tiles += tiles < 16 ? 1 : tiles / 4) {
            double all = n <= kOwnTokens ? kSortAndJoin : 0.0;
            for (int m = 0; m < d; ++m) all += work[m].of((double)n / tiles) * cdiv(combos * tiles, kSms) / d;
            if (all < least) {
                least = all;
                cs = c;
                for (int m = 0; m < d; ++m) st.tables[m] = t[m];
                st.s.tile = cdiv(n, tiles);
                st.s.tiles = cdiv(n, st.s.tile);
            }
        }
    }
    if (cs != 0) {
        st.s.a = a;
        st.stage = stage_args(a.index, a.factor, a.type, a.width);
        if (cs == 32) return grad_staged<32>(st, !quads, s);
        if (cs == 16) return grad_staged<16>(st, !quads, s);
        return grad_staged<8>(st, !quads, s);
    }
    if (a.type == MTTKRP_F32) return grad_cached<float>(a, s);
    if (a.type == MTTKRP_BF16) return grad_cached<__nv_bfloat16>(a, s);
    return grad_cached<__half>(a, s);
}

}  // namespace mk
