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

inline bool newton_some(const mttkrp_matrices& m) { return m.batch > 0 && m.rows > 0 && m.cols > 0; }
// whether newton_small.cu takes it: a short side of at most 128, and a long one that fits a cluster
bool newton_is_small(const mttkrp_matrices& m);
cudaError_t launch_newton_small(const NewtonArgs& a, int sms, cudaStream_t s);

// bytes for matrices of these shapes; 0 where none needs any
size_t newton_workspace_bytes(int n, const mttkrp_matrices* like);
cudaError_t launch_newton(const NewtonArgs& a, cudaStream_t s);

}  // namespace mk
