// q4_f32.cu -- the 4-bit matrix-vector kernel (q4.cuh) for x of type f32.
#include "q4.cuh"

namespace gbmm {

cudaError_t launch_q4_f32(const Q4Params &p, cudaStream_t s) { return q4::launch<q4::kFloat>(p, device_sm_count(), s); }

}  // namespace gbmm
