// Entry points of the operators of a sampled fit (include/mttkrp.h): checks on the host,
// then the launches of rows.cu, model.cu and gradnorm.cu.
#include <algorithm>
#include <memory>
#include <new>

#include "checks.h"
#include "rows.h"

namespace mk {
namespace {

constexpr int64_t kMaxTokens = INT32_MAX;
constexpr int64_t kMaxWidth = 65536;

int check_index(const void* idx, int64_t n, int64_t stride, int bytes) {
    if (bytes != 4 && bytes != 8) return fail(MTTKRP_ERR_INVALID, "indices of %d bytes: 4 or 8 are taken", bytes);
    if (n < 0 || n > kMaxTokens) return fail(MTTKRP_ERR_INVALID, "n=%lld outside [0, 2^31)", (long long)n);
    if (n > 0 && idx == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL indices");
    if (stride < 0) return fail(MTTKRP_ERR_INVALID, "negative index stride");
    if (!aligned_to(idx, bytes)) return fail(MTTKRP_ERR_INVALID, "indices must be %d-byte aligned", bytes);
    return MTTKRP_OK;
}

int check_rows(const char* what, const void* p, int64_t rows, int64_t width, int64_t stride, int type) {
    if (!type_ok(type)) return fail(MTTKRP_ERR_INVALID, "%s: unknown type %d", what, type);
    if (width < 1 || width > kMaxWidth)
        return fail(MTTKRP_ERR_INVALID, "width=%lld outside [1, %lld]", (long long)width, (long long)kMaxWidth);
    if (stride < width) return fail(MTTKRP_ERR_INVALID, "%s: rows closer than their width", what);
    if (stride > kMaxNumel || (rows > 0 && stride > kMaxNumel / rows))
        return fail(MTTKRP_ERR_INVALID, "%s spans more than 2^40 elements", what);
    if (rows > 0 && p == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL %s", what);
    if (!aligned_to(p, type_bytes(type)))
        return fail(MTTKRP_ERR_INVALID, "%s must be %zu-byte aligned", what, type_bytes(type));
    return MTTKRP_OK;
}

// a CP model and its coordinates; fills the index arguments
int check_model(int d, const int64_t* dims, int64_t R, const void* const* factors, int type, const void* coords,
                int64_t n, int idx_bytes, IndexArgs& index) {
    if (d < 1 || d > MTTKRP_MAX_ORDER) return fail(MTTKRP_ERR_INVALID, "order d=%d outside [1, %d]", d, MTTKRP_MAX_ORDER);
    if (dims == nullptr || factors == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL dims or factors");
    if (int rc = check_index(coords, n, d, idx_bytes)) return rc;
    if (R < 1 || R > kMaxR) return fail(MTTKRP_ERR_INVALID, "rank R=%lld outside [1, %lld]", (long long)R, (long long)kMaxR);
    index = IndexArgs{coords, idx_bytes, d, n, d, {}};
    for (int m = 0; m < d; ++m) {
        if (dims[m] < 1 || dims[m] > kMaxTokens)
            return fail(MTTKRP_ERR_INVALID, "dims[%d]=%lld outside [1, 2^31)", m, (long long)dims[m]);
        if (int rc = check_rows("factor", factors[m], dims[m], R, R, type)) return rc;
        index.rows[m] = dims[m];
    }
    return MTTKRP_OK;
}

// A result that overlaps another one, or a tensor that is not its own, would be written or
// read while another CTA writes it.  The results are put in order of their addresses, then
// every tensor looks among them; a result has its tensor's size, so that one that is its
// tensor cannot meet another result's (in_place: all are).
int check_disjoint(int n, const void* const* tensors, const int64_t* numels, const int* types, void* const* outs,
                   bool in_place) {
    struct Span {
        uintptr_t begin, end;
        int k;
    };
    constexpr int kFew = 512;
    Span few[kFew];
    std::unique_ptr<Span[]> many;
    if (n > kFew && !(many = std::unique_ptr<Span[]>(new (std::nothrow) Span[n])))
        return fail(MTTKRP_ERR_HOST_ALLOC, "no host memory to look at %d tensors", n);
    Span* const spans = many ? many.get() : few;
    int used = 0;
    for (int k = 0; k < n; ++k) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(outs[k]);
        if (numels[k] != 0) spans[used++] = Span{at, at + numels[k] * type_bytes(types[k]), k};
    }
    std::sort(spans, spans + used, [](const Span& a, const Span& b) { return a.begin < b.begin; });
    for (int i = 1; i < used; ++i)
        if (spans[i].begin < spans[i - 1].end)
            return fail(MTTKRP_ERR_INVALID, "results %d and %d overlap", std::min(spans[i - 1].k, spans[i].k),
                        std::max(spans[i - 1].k, spans[i].k));
    for (int k = 0; k < n && !in_place; ++k) {
        if (numels[k] == 0) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[k]), end = at + numels[k] * type_bytes(types[k]);
        // the last result that begins before the tensor's end
        const Span* s = std::lower_bound(spans, spans + used, end, [](const Span& a, uintptr_t x) { return a.begin < x; });
        if (s != spans && (--s)->end > at && s->k != k)
            return fail(MTTKRP_ERR_INVALID, "result %d overlaps tensor %d", s->k, k);
    }
    return MTTKRP_OK;
}

int check_tensors(int n, const void* const* tensors, const int64_t* numels, const int* types, void* const* outs,
                  const float* norm, const void* ws, size_t ws_bytes) {
    if (n < 0 || n > (1 << 20)) return fail(MTTKRP_ERR_INVALID, "n=%d tensors outside [0, 2^20]", n);
    if (n > 0 && (tensors == nullptr || numels == nullptr || types == nullptr))
        return fail(MTTKRP_ERR_INVALID, "NULL tensors, numels or types");
    if (norm == nullptr || !aligned_to(norm, 4)) return fail(MTTKRP_ERR_INVALID, "norm must be a 4-byte aligned pointer");
    int64_t total = 0;
    // Whether the results, and those tensors that are not their own results, are apart as most
    // lists are: the results one behind the other, the tensors outside of all they span.
    bool ascending = true, in_place = true;
    uintptr_t first = 0, behind = 0;
    for (int k = 0; k < n; ++k) {
        if (!type_ok(types[k])) return fail(MTTKRP_ERR_INVALID, "tensor %d: unknown type %d", k, types[k]);
        if (numels[k] < 0 || numels[k] > kMaxNumel - total)
            return fail(MTTKRP_ERR_INVALID, "tensor %d: %lld elements, or more than 2^40 in all", k, (long long)numels[k]);
        total += numels[k];
        if (numels[k] == 0) continue;
        const size_t e = type_bytes(types[k]);
        if (tensors[k] == nullptr || !aligned_to(tensors[k], e))
            return fail(MTTKRP_ERR_INVALID, "tensor %d: NULL or not %zu-byte aligned", k, e);
        if (outs == nullptr) continue;
        if (outs[k] == nullptr || !aligned_to(outs[k], e))
            return fail(MTTKRP_ERR_INVALID, "result %d: NULL or not %zu-byte aligned", k, e);
        if (outs[k] != tensors[k] && overlap(outs[k], numels[k] * e, tensors[k], numels[k] * e))
            return fail(MTTKRP_ERR_INVALID, "result %d overlaps its tensor without being it", k);
        const uintptr_t at = reinterpret_cast<uintptr_t>(outs[k]);
        first = behind == 0 ? at : first;
        ascending = ascending && at >= behind;
        behind = at + numels[k] * e;
        in_place = in_place && outs[k] == tensors[k];
    }
    bool outside = true;
    for (int k = 0; k < n && !in_place && ascending && outside; ++k)
        outside = !overlap(tensors[k], numels[k] * type_bytes(types[k]), reinterpret_cast<const void*>(first), behind - first);
    if (!ascending || !outside)
        if (int rc = check_disjoint(n, tensors, numels, types, outs, in_place)) return rc;
    return check_workspace(ws, ws_bytes, grad_norm_workspace_bytes(n));
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

int mttkrp_embedding(const void* table, int64_t rows, int64_t width, int64_t table_stride, int type, const void* idx,
                     int64_t n, int64_t idx_stride, int idx_bytes, float scale, void* out, int64_t out_stride,
                     void* stream) {
    clear_error();
    if (rows < 1 || rows > kMaxTokens) return fail(MTTKRP_ERR_INVALID, "rows=%lld outside [1, 2^31)", (long long)rows);
    if (int rc = check_index(idx, n, idx_stride, idx_bytes)) return rc;
    if (int rc = check_rows("table", table, rows, width, table_stride, type)) return rc;
    if (int rc = check_rows("result", out, n, width, out_stride, type)) return rc;
    const size_t e = type_bytes(type), no = span_bytes(n, width, out_stride, e);
    if (overlap(out, no, table, span_bytes(rows, width, table_stride, e)) ||
        overlap(out, no, idx, span_bytes(n, 1, idx_stride, idx_bytes)))
        return fail(MTTKRP_ERR_INVALID, "the result overlaps the table or the indices");
    LookupArgs a{table, table_stride, {idx, idx_bytes, idx_stride, n, 1, {rows}}, width, scale, out, out_stride};
    cudaError_t err = launch_lookup(a, type, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "lookup launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

size_t mttkrp_embedding_grad_workspace_bytes(int64_t n, int64_t rows, int64_t width) {
    if (n < 0 || n > kMaxTokens || rows < 1 || rows > kMaxTokens || width < 1 || width > kMaxWidth) return 0;
    return lookup_grad_workspace_bytes(IndexArgs{nullptr, 4, 1, n, 1, {rows}}, width);
}

int mttkrp_embedding_grad(const void* idx, int64_t n, int64_t idx_stride, int idx_bytes, const void* grad, int type,
                          int64_t grad_stride, int64_t rows, int64_t width, float scale, int accumulate, void* out,
                          int out_type, int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    if (rows < 1 || rows > kMaxTokens) return fail(MTTKRP_ERR_INVALID, "rows=%lld outside [1, 2^31)", (long long)rows);
    if (int rc = check_index(idx, n, idx_stride, idx_bytes)) return rc;
    if (int rc = check_rows("gradient", grad, n, width, grad_stride, type)) return rc;
    if (int rc = check_rows("result", out, rows, width, out_stride, out_type)) return rc;
    if (out_type != MTTKRP_F32 && out_type != type)
        return fail(MTTKRP_ERR_INVALID, "the result is in fp32 or in the gradient's type");
    const size_t no = span_bytes(rows, width, out_stride, type_bytes(out_type));
    if (overlap(out, no, grad, span_bytes(n, width, grad_stride, type_bytes(type))) ||
        overlap(out, no, idx, span_bytes(n, 1, idx_stride, idx_bytes)))
        return fail(MTTKRP_ERR_INVALID, "the result overlaps the gradient or the indices");
    RowSumArgs a{};
    a.index = IndexArgs{idx, idx_bytes, idx_stride, n, 1, {rows}};
    if (int rc = check_workspace(workspace, workspace_bytes, lookup_grad_workspace_bytes(a.index, width))) return rc;
    a.width = width;
    a.type = type;
    a.grad = grad;
    a.grad_stride = grad_stride;
    a.scale = scale;
    a.out[0] = out;
    a.out_stride = out_stride;
    a.out_type = out_type;
    a.accumulate = accumulate != 0;
    a.ws = workspace;
    cudaError_t err = launch_lookup_grad(a, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "lookup gradient launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

int mttkrp_cp_entries(int d, const int64_t* dims, int64_t R, const void* const* factors, int type, const void* coords,
                      int64_t n_samples, int idx_bytes, float* out, void* stream) {
    clear_error();
    EntriesArgs a{};
    if (int rc = check_model(d, dims, R, factors, type, coords, n_samples, idx_bytes, a.index)) return rc;
    if (n_samples > 0 && (out == nullptr || !aligned_to(out, 4)))
        return fail(MTTKRP_ERR_INVALID, "the result must be a 4-byte aligned pointer");
    for (int m = 0; m < d; ++m) {
        if (overlap(out, n_samples * 4, factors[m], span_bytes(dims[m], R, R, type_bytes(type))))
            return fail(MTTKRP_ERR_INVALID, "the result overlaps factor %d", m);
        a.factor[m] = factors[m];
    }
    if (overlap(out, n_samples * 4, coords, (size_t)n_samples * d * idx_bytes))
        return fail(MTTKRP_ERR_INVALID, "the result overlaps the coordinates");
    a.width = R;
    a.out = out;
    a.type = type;
    cudaError_t err = launch_entries(a, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "entries launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

size_t mttkrp_cp_entries_grad_workspace_bytes(int d, const int64_t* dims, int64_t R, int64_t n_samples) {
    if (d < 1 || d > MTTKRP_MAX_ORDER || dims == nullptr || R < 1 || R > kMaxR || n_samples < 0 || n_samples > kMaxTokens)
        return 0;
    IndexArgs index{nullptr, 4, d, n_samples, d, {}};
    for (int m = 0; m < d; ++m) {
        if (dims[m] < 1 || dims[m] > kMaxTokens) return 0;
        index.rows[m] = dims[m];
    }
    return entries_grad_workspace_bytes(index, R);
}

int mttkrp_cp_entries_grad(int d, const int64_t* dims, int64_t R, const void* const* factors, int type,
                           const void* coords, int64_t n_samples, int idx_bytes, const float* g, float* const* outs,
                           void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    RowSumArgs a{};
    if (int rc = check_model(d, dims, R, factors, type, coords, n_samples, idx_bytes, a.index)) return rc;
    if (outs == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL results");
    if (n_samples > 0 && (g == nullptr || !aligned_to(g, 4)))
        return fail(MTTKRP_ERR_INVALID, "the entries' gradient must be a 4-byte aligned pointer");
    for (int m = 0; m < d; ++m) {
        if (int rc = check_rows("result", outs[m], dims[m], R, R, MTTKRP_F32)) return rc;
        const size_t no = span_bytes(dims[m], R, R, 4);
        bool over = overlap(outs[m], no, coords, (size_t)n_samples * d * idx_bytes) ||
                    overlap(outs[m], no, g, (size_t)n_samples * 4);
        for (int l = 0; l < d; ++l) {
            over = over || overlap(outs[m], no, factors[l], span_bytes(dims[l], R, R, type_bytes(type)));
            over = over || (l < m && overlap(outs[m], no, outs[l], span_bytes(dims[l], R, R, 4)));
        }
        if (over) return fail(MTTKRP_ERR_INVALID, "result %d overlaps an input or another result", m);
        a.factor[m] = factors[m];
        a.out[m] = outs[m];
    }
    if (int rc = check_workspace(workspace, workspace_bytes, entries_grad_workspace_bytes(a.index, R))) return rc;
    a.width = R;
    a.type = type;
    a.g = g;
    a.scale = 1.f;
    a.out_stride = R;
    a.out_type = MTTKRP_F32;
    a.ws = workspace;
    cudaError_t err = launch_entries_grad(a, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "entries gradient launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

size_t mttkrp_grad_norm_workspace_bytes(int n) { return n < 0 || n > (1 << 20) ? 0 : grad_norm_workspace_bytes(n); }

int mttkrp_grad_norm(int n, const void* const* tensors, const int64_t* numels, const int* types, float* norm,
                     void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    if (int rc = check_tensors(n, tensors, numels, types, nullptr, norm, workspace, workspace_bytes)) return rc;
    cudaError_t err = launch_grad_norm(n, tensors, numels, types, nullptr, 0.f, 0.f, norm, workspace,
                                       static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "norm launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

int mttkrp_clip_grad_norm(int n, const void* const* tensors, const int64_t* numels, const int* types,
                          void* const* outs, float max_norm, float eps, float* norm, void* workspace,
                          size_t workspace_bytes, void* stream) {
    clear_error();
    if (outs == nullptr) outs = const_cast<void* const*>(tensors);   // in place: the tensors are the results
    if (!(max_norm >= 0.f) || !(eps >= 0.f)) return fail(MTTKRP_ERR_INVALID, "max_norm and eps must be >= 0");
    if (int rc = check_tensors(n, tensors, numels, types, outs, norm, workspace, workspace_bytes)) return rc;
    cudaError_t err = launch_grad_norm(n, tensors, numels, types,
                                       outs, max_norm, eps, norm, workspace, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "clipping launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

}  // extern "C"
