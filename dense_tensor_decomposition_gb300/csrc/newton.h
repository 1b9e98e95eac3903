// Orthogonalisation by Newton-Schulz products (newton.cu).  Nothing here is part of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "mttkrp.h"

namespace mk {

constexpr int kNewtonMaxSteps = 64;

// For matrix list element k, every matrix of it:
//   U = grad, or with momentum (M' = mu M + grad): grad + mu M' (nesterov), M'
//   out = alpha * weight + beta[k] * O(U)
struct NewtonArgs {
    int n;
    const mttkrp_matrices *grad, *momentum, *momentum_out, *weight, *out;   // HOST; momentum, weight: NULL for none
    float mu;
    bool nesterov;
    float alpha;
    const float* beta;          // n
    int steps;
    const float* coefficients;  // 3 a step
    double eps;
    void* ws;
    uint32_t* status;           // the device's error word
};

// bytes for matrices of these shapes; 0 where they cannot be taken
size_t newton_workspace_bytes(int n, const mttkrp_matrices* like);
cudaError_t launch_newton(const NewtonArgs& a, cudaStream_t s);

}  // namespace mk
