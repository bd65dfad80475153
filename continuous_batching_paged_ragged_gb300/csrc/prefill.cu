// The prefill tile kernel's instances for rows that see their whole context, and what the plan asks about it.
#include "prefill.cuh"

namespace pkv {

bool prefill_supported(int head_dim, int group) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         (group == 1 || group == 2 || group == 4 || group == 6 || group == 8);
}

int prefill_item_positions(int group, int head_dim) { return (head_dim == 256 ? 1 : kWG) * prefill_positions(group); }

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) { return launch_prefill_items<false>(a, stream); }

}  // namespace pkv
