// q4_run_f16.cu -- spmv_q4_run's kernels for f16 vectors.
#include "q4_run.cuh"

namespace spmv {
namespace q4 {
template cudaError_t launch_run<__half>(const RunArgs&, cudaStream_t);
}  // namespace q4
}  // namespace spmv
