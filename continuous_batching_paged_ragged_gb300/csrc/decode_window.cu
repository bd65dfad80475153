// The decode kernel's windowed instances for the fp16 cache: a token attends the last `window` keys of its context and
// its row's first `sinks`, and only the blocks holding those are streamed (see token_blocks).
#include "decode.cuh"

namespace pkv {

cudaError_t launch_decode_window(int head_dim, int group, const DecodeParams& p, pkv_pool* pool, int64_t max_tasks,
                                 cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_decode_g<64, kKvF16, true>(group, p, pool, max_tasks, stream);
    case 128: return launch_decode_g<128, kKvF16, true>(group, p, pool, max_tasks, stream);
    case 256: return launch_decode_g<256, kKvF16, true>(group, p, pool, max_tasks, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
