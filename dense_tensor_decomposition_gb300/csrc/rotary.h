// Rotation of rows by their position (rotary.cu).  Nothing here is part of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mttkrp.h"

namespace mk {

struct RotaryArgs {
    int n;                              // tensors
    const mttkrp_rotary_tensor* tensor; // HOST
    int type;
    int64_t batch, length, width;
    const void* positions;
    int pos_bytes;
    int64_t pos_batch_stride, pos_stride;
    int dims;
    const uint64_t* turns;              // HOST, dims / 2: turns a position, in 2^-64 of a turn
    bool interleaved, inverse;
    float scale;
};

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s);

}  // namespace mk
