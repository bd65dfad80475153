// The prefill tile kernel's windowed instances.
#include "prefill.cuh"

namespace pkv {

cudaError_t launch_prefill_window(const PrefillArgs& a, cudaStream_t stream) { return launch_prefill_items<true>(a, stream); }

}  // namespace pkv
