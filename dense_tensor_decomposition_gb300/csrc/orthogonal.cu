// Entry points of the orthogonal maps (include/mttkrp.h): checks on the host, then the
// launches of rotary.cu and newton.cu.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "checks.h"
#include "newton.h"
#include "rotary.h"
#include "tc.h"
#include "turns.h"

namespace mk {
namespace {

constexpr int64_t kMaxTokens = INT32_MAX;
constexpr int64_t kMaxWidth = 65536;

// Rows of `width` consecutive elements at all combinations of three indices.
struct Rows {
    uintptr_t at;
    int64_t extent[3], stride[3];       // stride in bytes, 0 where extent is 1
    int64_t width;                      // in bytes
    Rows(const void* p, int64_t batch, int64_t length, int64_t heads, const int64_t* strides, int64_t w, int64_t elem)
        : at(reinterpret_cast<uintptr_t>(p)), extent{batch, length, heads}, width(w * elem) {
        for (int m = 0; m < 3; ++m) stride[m] = extent[m] > 1 ? strides[m] * elem : 0;
    }
    bool empty() const { return extent[0] == 0 || extent[1] == 0 || extent[2] == 0; }
    // bytes from the first to behind the last, of the indices whose stride is below `period`
    int64_t span(int64_t period) const {
        int64_t bytes = width;
        for (int m = 0; m < 3; ++m)
            if (stride[m] < period) bytes += (extent[m] - 1) * stride[m];
        return bytes;
    }
    // whether every stride of at least `period` is a multiple of it
    bool repeats(int64_t period) const {
        for (int m = 0; m < 3; ++m)
            if (stride[m] >= period && stride[m] % period != 0) return false;
        return true;
    }
    // whether no element is met twice: each index steps over all that the smaller strides span
    bool apart() const {
        if (empty()) return true;
        for (int m = 0; m < 3; ++m) {
            if (extent[m] == 1) continue;
            int64_t below = width;
            for (int l = 0; l < 3; ++l)
                if (stride[l] < stride[m] || (stride[l] == stride[m] && l < m)) below += (extent[l] - 1) * stride[l];
            if (stride[m] < below) return false;
        }
        return true;
    }
};

// Whether two sets of rows can be told to share no byte: one lies behind the other, or both
// repeat with one period and lie apart within it (queries and keys in one buffer).
bool disjoint(const Rows& a, const Rows& b) {
    if (a.empty() || b.empty()) return true;
    const int64_t sa = a.span(INT64_MAX), sb = b.span(INT64_MAX);
    if (a.at + sa <= b.at || b.at + sb <= a.at) return true;
    for (int m = 0; m < 3; ++m) {
        const int64_t period = a.stride[m];
        if (period == 0 || !a.repeats(period) || !b.repeats(period)) continue;
        const int64_t from_a = (int64_t)((b.at - a.at) % (uintptr_t)period);
        const int64_t off = b.at >= a.at ? from_a : (period - (int64_t)((a.at - b.at) % (uintptr_t)period)) % period;
        if (off >= a.span(period) && off + b.span(period) <= period) return true;
    }
    return false;
}

int check_strides(const char* what, int k, const int64_t* extent, const int64_t* stride, int64_t width) {
    int64_t last = width;
    for (int m = 0; m < 3; ++m) {
        if (extent[m] <= 1) continue;
        if (stride[m] < 0) return fail(MTTKRP_ERR_INVALID, "%s %d: negative stride", what, k);
        if (stride[m] > (kMaxNumel - last) / (extent[m] - 1))
            return fail(MTTKRP_ERR_INVALID, "%s %d spans more than 2^40 elements", what, k);
        last += stride[m] * (extent[m] - 1);
    }
    return MTTKRP_OK;
}

constexpr int kMaxList = 1 << 20;
constexpr int64_t kMaxTiles = (int64_t)1 << 24;         // of one matrix's images

bool same_place(const mttkrp_matrices& a, const mttkrp_matrices& b) {
    return a.data == b.data && a.type == b.type && (a.batch <= 1 || a.batch_stride == b.batch_stride) &&
           (a.rows <= 1 || a.row_stride == b.row_stride);
}

bool none(const mttkrp_matrices& m) { return !newton_some(m); }

Rows rows_of(const mttkrp_matrices& m) {
    const int64_t strides[3] = {m.batch_stride, m.row_stride, 0};
    return Rows(m.data, m.batch, m.rows, 1, strides, m.cols, (int64_t)type_bytes(m.type));
}

int check_shapes(int n, const mttkrp_matrices* list) {
    if (n < 0 || n > kMaxList) return fail(MTTKRP_ERR_INVALID, "n=%d matrices outside [0, 2^20]", n);
    if (n > 0 && list == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL list");
    for (int k = 0; k < n; ++k) {
        const mttkrp_matrices& m = list[k];
        if (m.rows < 0 || m.rows > MTTKRP_MAX_NEWTON_SIDE || m.cols < 0 || m.cols > MTTKRP_MAX_NEWTON_SIDE ||
            m.batch < 0 || m.batch > kMaxTokens)
            return fail(MTTKRP_ERR_INVALID, "matrix %d: %lld x %lld x %lld out of range", k, (long long)m.batch,
                        (long long)m.rows, (long long)m.cols);
        const int64_t rt = (m.rows + 63) / 64, ct = (m.cols + 63) / 64, least = std::min(rt, ct);
        if (4 * (rt * ct + least * least) > kMaxTiles)
            return fail(MTTKRP_ERR_INVALID, "matrix %d: %lld x %lld needs more than 128 GB of images", k,
                        (long long)m.rows, (long long)m.cols);
    }
    return MTTKRP_OK;
}

int check_list(const char* what, int n, const mttkrp_matrices* list, const mttkrp_matrices* like) {
    if (n > 0 && list == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL %s", what);
    for (int k = 0; k < n; ++k) {
        const mttkrp_matrices& m = list[k];
        if (!type_ok(m.type)) return fail(MTTKRP_ERR_INVALID, "%s %d: unknown type %d", what, k, m.type);
        if (m.batch != like[k].batch || m.rows != like[k].rows || m.cols != like[k].cols)
            return fail(MTTKRP_ERR_INVALID, "%s %d: not of its matrix's shape", what, k);
        if (none(m)) continue;
        if (m.data == nullptr || !aligned_to(m.data, type_bytes(m.type)))
            return fail(MTTKRP_ERR_INVALID, "%s %d: NULL or not %zu-byte aligned", what, k, type_bytes(m.type));
        const int64_t extent[3] = {m.batch, m.rows, 1}, stride[3] = {m.batch_stride, m.row_stride, 0};
        if (int rc = check_strides(what, k, extent, stride, m.cols)) return rc;
        // (also where a result is written: every element once)
        if (m.rows > 1 && m.row_stride < m.cols) return fail(MTTKRP_ERR_INVALID, "%s %d: rows closer than their width", what, k);
        if (m.batch > 1 && m.batch_stride < (m.rows - 1) * m.row_stride + m.cols)
            return fail(MTTKRP_ERR_INVALID, "%s %d: matrices overlap", what, k);
    }
    return MTTKRP_OK;
}

// A list that is read, or written; an element of it may be written in the place of list number
// `place`'s (-1: of none).  (Not known by its address: a caller may pass one array as several lists.)
struct Listed {
    const char* what;
    const mttkrp_matrices* list;
    bool written;
    int place;
};

// No result overlaps another result or a tensor, but for its own place.
int check_apart(int n, const Listed* lists, int count) {
    struct Span {
        uintptr_t begin, end;
        int list, k;
    };
    const size_t most = (size_t)n * count;
    std::unique_ptr<Span[]> spans(new (std::nothrow) Span[most]);
    std::unique_ptr<size_t[]> open(new (std::nothrow) size_t[most]);
    if (!spans || !open) return fail(MTTKRP_ERR_HOST_ALLOC, "no host memory to look at %d matrices", n);
    size_t used = 0;
    for (int l = 0; l < count; ++l)
        for (int k = 0; k < n; ++k) {
            const mttkrp_matrices& m = lists[l].list[k];
            if (none(m)) continue;
            const Rows r = rows_of(m);
            spans[used++] = Span{r.at, r.at + (uintptr_t)r.span(INT64_MAX), l, k};
        }
    std::sort(spans.get(), spans.get() + used, [](const Span& a, const Span& b) { return a.begin < b.begin; });
    size_t opened = 0;          // spans that end behind where the present one begins
    for (size_t i = 0; i < used; ++i) {
        const Span& x = spans[i];
        size_t kept = 0;
        for (size_t o = 0; o < opened; ++o) {
            const Span& y = spans[open[o]];
            if (y.end <= x.begin) continue;
            open[kept++] = open[o];
            const Listed &lx = lists[x.list], &ly = lists[y.list];
            if (!lx.written && !ly.written) continue;
            const mttkrp_matrices &mx = lx.list[x.k], &my = ly.list[y.k];
            if (x.k == y.k && (lx.place == y.list || ly.place == x.list) && same_place(mx, my)) continue;
            if (!disjoint(rows_of(mx), rows_of(my)))
                return fail(MTTKRP_ERR_INVALID, "%s %d overlaps %s %d", lx.what, x.k, ly.what, y.k);
        }
        opened = kept;
        open[opened++] = i;
    }
    return MTTKRP_OK;
}

// the largest magnitude of s (a + b s^2 + c s^4) for s in [0, most], and of the bracket
void reach(const double* abc, double most, double& value, double& bracket) {
    const double a = abc[0], b = abc[1], c = abc[2], top = most * most;
    bracket = std::max(std::fabs(a), std::fabs(a + top * (b + top * c)));
    value = most * std::fabs(a + top * (b + top * c));
    if (c != 0.0) {
        const double turn = -b / (2.0 * c);
        if (turn > 0.0 && turn < top) bracket = std::max(bracket, std::fabs(a + turn * (b + turn * c)));
    }
    // a + 3 b z + 5 c z^2 = 0, z = s^2
    double z[2] = {-1.0, -1.0};
    const double square = 9.0 * b * b - 20.0 * a * c;
    if (c != 0.0 && square >= 0.0) {
        z[0] = (-3.0 * b + std::sqrt(square)) / (10.0 * c);
        z[1] = (-3.0 * b - std::sqrt(square)) / (10.0 * c);
    } else if (c == 0.0 && b != 0.0) {
        z[0] = -a / (3.0 * b);
    }
    for (const double at : z)
        if (at > 0.0 && at < top) value = std::max(value, std::sqrt(at) * std::fabs(a + at * (b + at * c)));
}

int check_steps(int steps, const double* coefficients, double eps, float* rounded) {
    if (steps < 1 || steps > MTTKRP_MAX_NEWTON_STEPS)
        return fail(MTTKRP_ERR_INVALID, "steps=%d outside [1, %d]", steps, MTTKRP_MAX_NEWTON_STEPS);
    if (coefficients == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL coefficients");
    if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(MTTKRP_ERR_INVALID, "eps must be finite and >= 0");
    double most = 1.0;          // of the singular values
    for (int i = 0; i < steps; ++i) {
        double bracket = 0.0, value = 0.0;
        for (int e = 0; e < 3; ++e)
            if (!std::isfinite(coefficients[3 * i + e])) return fail(MTTKRP_ERR_INVALID, "coefficients of step %d are not finite", i);
        reach(coefficients + 3 * i, most, value, bracket);
        if (!(bracket <= 15.9))
            return fail(MTTKRP_ERR_INVALID, "step %d: its coefficients multiply a singular value by %.3g, above 15.9", i, bracket);
        if (!(value <= 3.9) && i + 1 < steps)
            return fail(MTTKRP_ERR_INVALID, "step %d: its coefficients let a singular value grow to %.3g, above 3.9", i, value);
        most = value;
        for (int e = 0; e < 3; ++e) rounded[3 * i + e] = (float)coefficients[3 * i + e];
    }
    return MTTKRP_OK;
}

int run_newton(NewtonArgs& a, const float* scales, double factor, void* ws, size_t ws_bytes, void* stream) {
    if (int rc = check_workspace(ws, ws_bytes, newton_workspace_bytes(a.n, a.grad))) return rc;
    int some = 0;
    for (int k = 0; k < a.n; ++k) some += newton_some(a.grad[k]);
    if (some == 0) return MTTKRP_OK;
    std::unique_ptr<float[]> beta(new (std::nothrow) float[a.n]);
    if (!beta) return fail(MTTKRP_ERR_HOST_ALLOC, "no host memory for %d scales", a.n);
    for (int k = 0; k < a.n; ++k) beta[k] = (float)(factor * (scales ? (double)scales[k] : 1.0));
    a.beta = beta.get();
    a.ws = ws;
    a.status = tc_status_ptr();
    if (a.status == nullptr) return fail(MTTKRP_ERR_CUDA, "device status word unavailable");
    cudaError_t err = launch_newton(a, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "orthogonalisation launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

int mttkrp_rotary(int n, const mttkrp_rotary_tensor* tensors, int type, int64_t batch, int64_t length, int64_t width,
                  const void* positions, int pos_bytes, int64_t pos_batch_stride, int64_t pos_stride,
                  const double* frequencies, int dims, int interleaved, float scale, int inverse, void* stream) {
    clear_error();
    if (n < 1 || n > MTTKRP_MAX_ROTARY) return fail(MTTKRP_ERR_INVALID, "n=%d tensors outside [1, %d]", n, MTTKRP_MAX_ROTARY);
    if (tensors == nullptr || frequencies == nullptr) return fail(MTTKRP_ERR_INVALID, "NULL tensors or frequencies");
    if (!type_ok(type)) return fail(MTTKRP_ERR_INVALID, "unknown type %d", type);
    if (batch < 0 || length < 0 || batch > kMaxTokens || length > kMaxTokens ||
        (length > 0 && batch > kMaxTokens / length))
        return fail(MTTKRP_ERR_INVALID, "%lld x %lld tokens: none to 2^31 - 1 are taken", (long long)batch, (long long)length);
    if (width < 1 || width > kMaxWidth)
        return fail(MTTKRP_ERR_INVALID, "width=%lld outside [1, %lld]", (long long)width, (long long)kMaxWidth);
    if (dims < 2 || dims > MTTKRP_MAX_ROTARY_DIMS || dims % 2 != 0 || dims > width)
        return fail(MTTKRP_ERR_INVALID, "dims=%d must be even, in [2, %d] and not above the width", dims,
                    MTTKRP_MAX_ROTARY_DIMS);
    if (pos_bytes != 4 && pos_bytes != 8) return fail(MTTKRP_ERR_INVALID, "positions of %d bytes: 4 or 8 are taken", pos_bytes);
    const int64_t tokens = batch * length;
    if (tokens > 0 && (positions == nullptr || !aligned_to(positions, pos_bytes)))
        return fail(MTTKRP_ERR_INVALID, "positions must be a %d-byte aligned pointer", pos_bytes);
    const int64_t pos_extent[3] = {batch, length, 1}, pos_strides[3] = {pos_batch_stride, pos_stride, 0};
    if (int rc = check_strides("positions", 0, pos_extent, pos_strides, 1)) return rc;
    uint64_t turns[MTTKRP_MAX_ROTARY_DIMS / 2];
    for (int i = 0; i < dims / 2; ++i) {
        if (!std::isfinite(frequencies[i])) return fail(MTTKRP_ERR_INVALID, "frequency %d is not finite", i);
        if (std::fabs(frequencies[i]) >= kMostRadians)
            return fail(MTTKRP_ERR_INVALID, "frequency %d: 2^64 radians a position or more", i);
        turns[i] = turns_of(frequencies[i]);
    }
    const int64_t e = (int64_t)type_bytes(type);
    mttkrp_rotary_tensor list[MTTKRP_MAX_ROTARY];
    int64_t heads = 0;
    const Rows where(positions, batch, length, 1, pos_strides, 1, pos_bytes);
    for (int k = 0; k < n; ++k) {
        list[k] = tensors[k];
        mttkrp_rotary_tensor& t = list[k];
        if (t.heads < 0 || t.heads > kMaxTokens - heads)
            return fail(MTTKRP_ERR_INVALID, "tensor %d: %lld heads", k, (long long)t.heads);
        heads += t.heads;
        if (t.heads == 0 || tokens == 0) continue;
        if (t.x == nullptr || t.out == nullptr || !aligned_to(t.x, e) || !aligned_to(t.out, e))
            return fail(MTTKRP_ERR_INVALID, "tensor %d or its result: NULL or not %d-byte aligned", k, (int)e);
        const int64_t extent[3] = {batch, length, t.heads};
        for (int m = 0; m < 3; ++m)
            if (extent[m] == 1) t.x_strides[m] = t.out_strides[m] = 0;
        if (int rc = check_strides("tensor", k, extent, t.x_strides, width)) return rc;
        if (int rc = check_strides("result", k, extent, t.out_strides, width)) return rc;
        const Rows out(t.out, batch, length, t.heads, t.out_strides, width, e);
        if (!out.apart()) return fail(MTTKRP_ERR_INVALID, "result %d: its rows overlap", k);
        if (!disjoint(where, out)) return fail(MTTKRP_ERR_INVALID, "result %d overlaps the positions", k);
        bool same = t.x == t.out;
        for (int m = 0; m < 3; ++m) same = same && t.x_strides[m] == t.out_strides[m];
        if (!same && !disjoint(Rows(t.x, batch, length, t.heads, t.x_strides, width, e), out))
            return fail(MTTKRP_ERR_INVALID, "result %d overlaps its tensor without being it", k);
        for (int l = 0; l < k; ++l) {
            const mttkrp_rotary_tensor& o = list[l];
            if (o.heads == 0) continue;
            const Rows other_x(o.x, batch, length, o.heads, o.x_strides, width, e);
            const Rows other(o.out, batch, length, o.heads, o.out_strides, width, e);
            if (!disjoint(other, out)) return fail(MTTKRP_ERR_INVALID, "results %d and %d overlap", l, k);
            if (!disjoint(other_x, out)) return fail(MTTKRP_ERR_INVALID, "result %d overlaps tensor %d", k, l);
            if (!disjoint(other, Rows(t.x, batch, length, t.heads, t.x_strides, width, e)))
                return fail(MTTKRP_ERR_INVALID, "result %d overlaps tensor %d", l, k);
        }
    }
    int used = 0;
    for (int k = 0; k < n; ++k)
        if (list[k].heads > 0) list[used++] = list[k];
    if (used == 0 || tokens == 0) return MTTKRP_OK;
    const RotaryArgs a{used, list, type, batch, length, width, positions, pos_bytes,
                       batch > 1 ? pos_batch_stride : 0, length > 1 ? pos_stride : 0,
                       dims, turns, interleaved != 0, inverse != 0, scale};
    cudaError_t err = launch_rotary(a, static_cast<cudaStream_t>(stream));
    if (err == cudaErrorInvalidConfiguration) return fail(MTTKRP_ERR_INVALID, "more vectors than a grid can hold");
    if (err != cudaSuccess) return fail(MTTKRP_ERR_CUDA, "rotation launch: %s", cudaGetErrorString(err));
    return MTTKRP_OK;
}

size_t mttkrp_orthogonalize_workspace_bytes(int n, const mttkrp_matrices* in) {
    clear_error();
    return check_shapes(n, in) == MTTKRP_OK ? newton_workspace_bytes(n, in) : 0;
}

int mttkrp_orthogonalize(int n, const mttkrp_matrices* in, const mttkrp_matrices* out, int steps,
                         const double* coefficients, double eps, const float* scales, void* workspace,
                         size_t workspace_bytes, void* stream) {
    clear_error();
    float abc[3 * MTTKRP_MAX_NEWTON_STEPS];
    if (int rc = check_shapes(n, in)) return rc;
    if (int rc = check_list("matrix", n, in, in)) return rc;
    if (int rc = check_list("result", n, out, in)) return rc;
    if (int rc = check_steps(steps, coefficients, eps, abc)) return rc;
    const Listed lists[2] = {{"matrix", in, false, -1}, {"result", out, true, 0}};
    if (int rc = check_apart(n, lists, 2)) return rc;
    NewtonArgs a{};
    a.n = n;
    a.grad = in;
    a.out = out;
    a.steps = steps;
    a.coefficients = abc;
    a.eps = eps;
    return run_newton(a, scales, 1.0, workspace, workspace_bytes, stream);
}

int mttkrp_orthogonal_step(int n, const mttkrp_matrices* weights, const mttkrp_matrices* grads,
                           const mttkrp_matrices* momenta, const mttkrp_matrices* weights_out,
                           const mttkrp_matrices* momenta_out, double lr, double momentum, int nesterov,
                           double weight_decay, int steps, const double* coefficients, double eps,
                           const float* scales, void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    float abc[3 * MTTKRP_MAX_NEWTON_STEPS];
    if (int rc = check_shapes(n, grads)) return rc;
    if (int rc = check_list("gradient", n, grads, grads)) return rc;
    if (int rc = check_list("weight", n, weights, grads)) return rc;
    if (int rc = check_list("momentum", n, momenta, grads)) return rc;
    if (int rc = check_list("new weight", n, weights_out, grads)) return rc;
    if (int rc = check_list("new momentum", n, momenta_out, grads)) return rc;
    for (int k = 0; k < n; ++k)
        if (weights[k].type != weights_out[k].type || momenta[k].type != momenta_out[k].type)
            return fail(MTTKRP_ERR_INVALID, "result %d is not of its tensor's type", k);
    if (!std::isfinite(lr) || !std::isfinite(momentum) || !std::isfinite(weight_decay))
        return fail(MTTKRP_ERR_INVALID, "lr, momentum and weight_decay must be finite");
    if (int rc = check_steps(steps, coefficients, eps, abc)) return rc;
    const Listed lists[5] = {{"gradient", grads, false, -1}, {"weight", weights, false, -1}, {"momentum", momenta, false, -1},
                             {"new weight", weights_out, true, 1}, {"new momentum", momenta_out, true, 2}};
    if (int rc = check_apart(n, lists, 5)) return rc;
    NewtonArgs a{};
    a.n = n;
    a.grad = grads;
    a.momentum = momenta;
    a.momentum_out = momenta_out;
    a.weight = weights;
    a.out = weights_out;
    a.mu = (float)momentum;
    a.nesterov = nesterov != 0;
    a.alpha = (float)(1.0 - lr * weight_decay);
    a.steps = steps;
    a.coefficients = abc;
    a.eps = eps;
    return run_newton(a, scales, -lr, workspace, workspace_bytes, stream);
}

}  // extern "C"
