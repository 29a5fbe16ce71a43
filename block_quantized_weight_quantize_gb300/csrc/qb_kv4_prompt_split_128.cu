// qb_kv4_prompt_split_128.cu -- the prompt kernel for calls with trees or sinks whose sequences have few
// rows, heads of up to 128 elements.
#include "qb_kv4_prompt.cuh"

namespace qb {
int launch_kv4_prompt_split_128(const Kv4AttnArgs &a, cudaStream_t stream) { return launch_kv4_prompt<128, true, true>(a, stream); }
}  // namespace qb
