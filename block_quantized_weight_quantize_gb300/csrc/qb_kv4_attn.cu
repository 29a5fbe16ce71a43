// qb_kv4_attn.cu -- attention over the paged 4-bit cache (qgemv.h: kv4_attn):
// which kernel takes a call, and the workspace.
#include <algorithm>
#include <cstdint>

#include "qb_kv4_prompt.cuh"
#include "qb_kv4_step.cuh"

namespace qb {

int64_t kv4_attn_ws(int dp) {
    int64_t most = 0;
    for (int pair = 0; pair < 2; ++pair)
        most = std::max(most, step_ws(attn_grid(), step_warps(dp), step_rows(pair != 0), dp).end);
    if (dp <= 128) most = std::max(most, prompt_ws(attn_grid(), dp).end);
    return most;
}

// Rows (token, query head) a sequence and key head, on average, from which the
// prompt kernel takes a half-precision call: its items have 256 rows, the step
// kernel's 8, which read and decode the keys anew.  Step against prompt kernel, us,
// heads of 128, 32 on 8 key heads, in bf16, every sequence with as many rows:
//     rows                        64          96          128         192
//     1 sequence of 2000 keys     18 / 36     21 / 35     23 / 36     27 / 36
//     1 of 8000                   30 / 33     39 / 33     46 / 33     62 / 33
//     8 of 2000                   50 / 52     66 / 52     83 / 52     117 / 52
//     8 of 8000                   141 / 86    203 / 87    265 / 88    389 / 89
//     64 of 300                   72 / 86     124 / 82    132 / 80    197 / 91
//     64 of 2000                  284 / 241   402 / 242   530 / 248   781 / 250
// The rule takes the slower kernel where one short sequence fills little of the card
// (from 96 rows) and where much work has 64 to 95 rows.
constexpr int kPromptFrom = 96;

int launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t stream) {
    if (a.type != QB_T_F32 && a.c.dp <= 128 && a.ntok * (a.nh / a.c.nkv) >= (int64_t)kPromptFrom * a.s.nseq)
        return a.c.dp == 64 ? launch_kv4_prompt_64(a, stream) : launch_kv4_prompt_128(a, stream);
    return a.c.dp == 64 ? launch_kv4_step_64(a, stream)
           : a.c.dp == 128 ? launch_kv4_step_128(a, stream) : launch_kv4_step_256(a, stream);
}

}  // namespace qb
