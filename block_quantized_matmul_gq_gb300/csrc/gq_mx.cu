// gq_mx.cu -- the microscaled mul_mat: MXFP4 weights times X quantized to MXFP4.
#include "gq_internal.h"

namespace gq {

int64_t mx4x_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    (void)M;
    return few_mx_workspace_bytes(K, N);
}

cudaError_t launch_mx4x(const MatProblem& p, int64_t N, void* workspace, cudaStream_t s) {
    return launch_few_mx4x(p, N, workspace, s);
}

}  // namespace gq
