// qb_kv4_step_ext_128.cu -- the step kernel for calls with trees or sinks, heads of up to 128 elements.
#include <algorithm>

#include "qb_kv4_step.cuh"

namespace qb {
int launch_kv4_step_ext_128(const Kv4AttnArgs &a, cudaStream_t stream) { return launch_kv4_step<128, true>(a, stream); }
}  // namespace qb
