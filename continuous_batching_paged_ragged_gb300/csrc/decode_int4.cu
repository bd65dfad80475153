// The decode kernel's 4-bit cache instances (codes with a scale for every 32 values), compiled apart from the others so
// that the sets build in parallel.
#include "decode_int4.cuh"

namespace pkv {

cudaError_t launch_decode_int4(int head_dim, int group, const DecodeParams& p, pkv_pool* pool, int64_t max_tasks,
                               cudaStream_t stream) {
  return launch_int4_shape<false>(head_dim, group, p, pool, max_tasks, stream);
}

}  // namespace pkv
