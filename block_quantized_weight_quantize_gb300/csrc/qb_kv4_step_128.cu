// qb_kv4_step_128.cu -- the step kernel of the 4-bit cache's attention for heads of up to 128 elements.
#include <algorithm>

#include "qb_kv4_step.cuh"

namespace qb {
int launch_kv4_step_128(const Kv4AttnArgs &a, cudaStream_t stream) { return launch_kv4_step<128>(a, stream); }
}  // namespace qb
