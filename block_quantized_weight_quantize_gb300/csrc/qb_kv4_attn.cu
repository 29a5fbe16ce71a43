// qb_kv4_attn.cu -- attention over the paged 4-bit cache (qgemv.h: kv4_attn):
// which kernel takes a call, and the workspace.
#include <algorithm>
#include <cstdint>

#include "qb_kv4_prompt.cuh"
#include "qb_kv4_step.cuh"

namespace qb {

int64_t kv4_attn_ws(int dp) {
    int64_t most = 0;
    for (int nt = 1; nt <= 2; ++nt)
        for (int pair = 0; pair < 2; ++pair)
            most = std::max(most, step_ws(attn_grid(), step_warps(dp, pair != 0, nt), step_rows(pair != 0, nt), dp).end);
    if (dp <= 128) most = std::max(most, prompt_ws(attn_grid(), dp).end);
    return most;
}

// Rows (token, query head) a sequence and key head, on average, from which the
// prompt kernel takes a half-precision call.
constexpr int kPromptFrom = 64;

int launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t stream) {
    if (a.type != QB_T_F32 && a.c.dp <= 128 && a.ntok * (a.nh / a.c.nkv) >= (int64_t)kPromptFrom * a.s.nseq)
        return a.c.dp == 64 ? launch_kv4_prompt_64(a, stream) : launch_kv4_prompt_128(a, stream);
    return a.c.dp == 64 ? launch_kv4_step_64(a, stream)
           : a.c.dp == 128 ? launch_kv4_step_128(a, stream) : launch_kv4_step_256(a, stream);
}

}  // namespace qb
