// Operators on rows of tables: lookup of a table's rows and its gradient by sorted
// tokens (rows.cu), the entries of a CP model at coordinates and the gradient of
// every factor (model.cu), norm and clipping (gradnorm.cu).  Nothing here is part of
// the C ABI.
//
// Where an index is outside its table the token (or sample) takes no part.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "mttkrp.h"

namespace mk {

// Indices of n tokens into d tables: token t's index into table m sits at
// element t * stride + m.  d = 1 for a lookup, the tensor's order for a CP model.
struct IndexArgs {
    const void* idx;
    int bytes;          // 4 or 8 an index
    int64_t stride;
    int64_t n;
    int d;
    int64_t rows[MTTKRP_MAX_ORDER];
};

struct LookupArgs {
    const void* table;
    int64_t table_stride;   // in elements
    IndexArgs index;
    int64_t width;
    float scale;
    void* out;
    int64_t out_stride;
};

// Sums of rows over the tokens of each index: for table m,
//   out[m][v, :] (+)= scale * sum over tokens t with index v of row(m, t, :)
// row = grad[t, :] for a lookup's gradient, or
// g[t] * prod over l != m of factor[l][idx(t, l), :] for a CP model's.
struct RowSumArgs {
    IndexArgs index;
    int64_t width;
    int type;               // of grad or the factors (MTTKRP_F32, ...)
    const void* grad;
    int64_t grad_stride;
    const void* factor[MTTKRP_MAX_ORDER];
    const float* g;
    float scale;
    void* out[MTTKRP_MAX_ORDER];
    int64_t out_stride;
    int out_type;           // MTTKRP_F32 or `type`
    int accumulate;
    void* ws;
};

struct EntriesArgs {
    IndexArgs index;
    int64_t width;
    int type;
    const void* factor[MTTKRP_MAX_ORDER];
    float* out;
};

cudaError_t launch_lookup(const LookupArgs& a, int type, cudaStream_t s);
cudaError_t launch_lookup_grad(const RowSumArgs& a, cudaStream_t s);
size_t lookup_grad_workspace_bytes(const IndexArgs& index, int64_t width);

cudaError_t launch_entries(const EntriesArgs& a, cudaStream_t s);
size_t entries_grad_workspace_bytes(const IndexArgs& index, int64_t width);
cudaError_t launch_entries_grad(const RowSumArgs& a, cudaStream_t s);

// Norm over many tensors and clipping by it (gradnorm.cu).  outs = nullptr: the
// norm alone.
size_t grad_norm_workspace_bytes(int n);
cudaError_t launch_grad_norm(int n, const void* const* tensors, const int64_t* numels, const int* types,
                             void* const* outs, float max_norm, float eps, float* norm, void* ws,
                             cudaStream_t s);

}  // namespace mk
