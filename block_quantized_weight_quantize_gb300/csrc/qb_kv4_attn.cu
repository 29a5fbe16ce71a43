// qb_kv4_attn.cu -- attention over the paged 4-bit cache (qgemv.h: kv4_attn):
// which kernel takes a call, and the workspace.
#include <algorithm>
#include <cstdint>

#include "qb_kv4_step.cuh"

namespace qb {

int64_t kv4_attn_ws(int nkv, int dp, int nh) {
    (void)nkv;
    (void)nh;
    const int64_t workers = (int64_t)std::min(num_sms(), 256) * kStepWarps;
    return workers * 2 * kMaxRows * (4 * dp + 8) + workers * 2 * 16;
}

int launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t stream) {
    return a.c.dp == 64 ? launch_kv4_step_64(a, stream)
           : a.c.dp == 128 ? launch_kv4_step_128(a, stream) : launch_kv4_step_256(a, stream);
}

}  // namespace qb
