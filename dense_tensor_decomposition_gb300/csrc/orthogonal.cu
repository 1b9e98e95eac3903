// Entry points of the orthogonal maps (include/mttkrp.h): checks on the host, then the
// launches of rotary.cu.
#include <cmath>

#include "checks.h"
#include "rotary.h"

namespace mk {
namespace {

constexpr int64_t kMaxTokens = INT32_MAX;
constexpr int64_t kMaxWidth = 65536;
constexpr double kTwoPi = 6.283185307179586476925286766559;

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
        double f = frequencies[i] / kTwoPi;
        f -= std::floor(f);                             // in [0, 1]: a whole turn more changes nothing
        turns[i] = f < 1.0 ? (uint64_t)std::ldexp(f, 64) : 0;
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

}  // extern "C"
