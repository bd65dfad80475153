// The decode kernel's windowed instances for the 4-bit cache: a token attends the last `window` keys of its context and
// its row's first `sinks`, and only the blocks holding those are streamed (see token_blocks).
#include "decode_int4.cuh"

namespace pkv {

cudaError_t launch_decode_window_int4(int head_dim, int group, const DecodeParams& p, pkv_pool* pool, int64_t max_tasks,
                                      cudaStream_t stream) {
  return launch_int4_shape<true>(head_dim, group, p, pool, max_tasks, stream);
}

}  // namespace pkv
