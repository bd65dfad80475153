// The decode kernel's windowed instances for the 4-bit cache: a token attends the last `window` keys of its context and
// its row's first `sinks`, and only the blocks holding those are streamed (see token_blocks).
#include "decode_int4.cuh"

namespace pkv {

cudaError_t launch_decode_window_int4(int head_dim, int group, const DecodeParams& p, pkv_pool* pool, int64_t max_tasks,
                                      cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_decode_g<64, kKvInt4, true>(group, p, pool, max_tasks, stream);
    case 128: return launch_decode_g<128, kKvInt4, true>(group, p, pool, max_tasks, stream);
    case 256: return launch_decode_g<256, kKvInt4, true>(group, p, pool, max_tasks, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
