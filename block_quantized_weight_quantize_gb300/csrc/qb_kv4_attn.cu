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
// With trees or sinks, where items' own cost is weighed and row tiles share the key tiles of few rows: step against
// prompt kernel, us, trees of rows / 4 tokens, otherwise as above:
//     rows                        32          48          64          96          128
//     1 sequence of 2000 keys     18 / 34     18 / 35     19 / 35     23 / 35     25 / 35
//     1 of 8000                   25 / 31     28 / 31     32 / 31     40 / 31     48 / 32
//     8 of 300                    18 / 25     21 / 25     25 / 25     30 / 25     42 / 26
//     8 of 2000                   34 / 45     42 / 45     51 / 45     70 / 45     86 / 46
//     8 of 8000                   79 / 69     110 / 69    139 / 69    200 / 70    260 / 70
//     32 of 1000                  62 / 74     95 / 74     116 / 74    154 / 74    202 / 75
//     64 of 300                   52 / 71     66 / 71     81 / 71     131 / 71    133 / 73
//     64 of 2000                  155 / 205   218 / 209   284 / 207   407 / 205   534 / 210
// Row tiles share key tiles (twice 128 rows take 250 us of the last line instead) where an average sequence's rows
// fill one.
constexpr int kPromptExtFrom = 40, kPromptExtMid = 48, kPromptSplitTo = 128;

int launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t stream) {
    if (kv4_attn_ext(a)) {
        const int64_t rows = a.ntok * (a.nh / a.c.nkv), items = (int64_t)a.s.nseq * a.c.nkv;
        const int64_t from = items >= num_sms() ? kPromptExtFrom : 3 * items >= num_sms() ? kPromptExtMid : kPromptFrom;
        if (a.type != QB_T_F32 && a.c.dp <= 128 && rows >= from * a.s.nseq) {
            if (rows <= (int64_t)kPromptSplitTo * a.s.nseq)
                return a.c.dp == 64 ? launch_kv4_prompt_split_64(a, stream) : launch_kv4_prompt_split_128(a, stream);
            return a.c.dp == 64 ? launch_kv4_prompt_ext_64(a, stream) : launch_kv4_prompt_ext_128(a, stream);
        }
        return a.c.dp == 64 ? launch_kv4_step_ext_64(a, stream)
               : a.c.dp == 128 ? launch_kv4_step_ext_128(a, stream) : launch_kv4_step_ext_256(a, stream);
    }
    if (a.type != QB_T_F32 && a.c.dp <= 128 && a.ntok * (a.nh / a.c.nkv) >= (int64_t)kPromptFrom * a.s.nseq)
        return a.c.dp == 64 ? launch_kv4_prompt_64(a, stream) : launch_kv4_prompt_128(a, stream);
    return a.c.dp == 64 ? launch_kv4_step_64(a, stream)
           : a.c.dp == 128 ? launch_kv4_step_128(a, stream) : launch_kv4_step_256(a, stream);
}

}  // namespace qb
