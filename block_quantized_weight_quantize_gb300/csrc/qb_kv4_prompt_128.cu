// qb_kv4_prompt_128.cu -- the prompt kernel of the 4-bit cache's attention for heads of up to 128 elements.
#include "qb_kv4_prompt.cuh"

namespace qb {
int launch_kv4_prompt_128(const Kv4AttnArgs &a, cudaStream_t stream) { return launch_kv4_prompt<128>(a, stream); }
}  // namespace qb
