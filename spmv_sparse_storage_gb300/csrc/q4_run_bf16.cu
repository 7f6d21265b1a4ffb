// q4_run_bf16.cu -- spmv_q4_run's kernels for bf16 vectors.
#include "q4_run.cuh"

namespace spmv {
namespace q4 {
template cudaError_t launch_run<__nv_bfloat16>(const RunArgs&, cudaStream_t);
}  // namespace q4
}  // namespace spmv
