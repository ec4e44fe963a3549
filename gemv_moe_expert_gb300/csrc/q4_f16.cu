// q4_f16.cu -- the 4-bit matrix-vector kernel (q4.cuh) for x of type f16.
#include "q4.cuh"

namespace gbmm {

cudaError_t launch_q4_f16(const Q4Params &p, cudaStream_t s) { return q4::launch<q4::kHalf>(p, device_sm_count(), s); }

}  // namespace gbmm
