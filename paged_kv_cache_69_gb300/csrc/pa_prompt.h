// pa_prompt.h -- host side of the prompt kernel: what pa_prefill.cu offers to
// the calls that launch it.
#pragma once

#include <cstddef>

#include "pa_common.h"

namespace pa {

struct PromptCall {
    const char* who;                   // call named in error details
    void* out;
    const void* q;
    pa_dtype dtype;                    // of q, out, K and V
    const void *k, *v;                 // contiguous rows (k_start) or pools (block_tables)
    const int32_t *q_start, *k_start, *seq_lens, *block_tables;
    int B, Hq, Hkv, D, total_q, total_k, bs, NB, MB;
    float scale;
    bool shared;                       // q_start: members of groups, seq_lens: prefixes; partials only
    const int32_t* lens;               // shared: lengths of the sequences
    int32_t *tail_lens, *tail_blk;     // shared: out
    int32_t* err_flag;
    cudaStream_t stream;
};

// How a call may be cut: the most ranges of keys per item and the partials' room.
struct PromptPlan {
    int grid = 1, splits = 1;
    size_t cut_bytes = 0, ml_bytes = 0, acc_bytes = 0;     // 0 without partials
    size_t bytes() const { return cut_bytes + ml_bytes + acc_bytes; }
};
PromptPlan prompt_plan(int B, int total_q, int Hq, int Hkv, int D, int max_keys, bool prompts, bool shared,
                       int sms);
// Room for any call of at most these numbers (a workspace made once serves smaller calls).
size_t prompt_part_bytes(int total_q, int Hq, int D, bool shared, int sms);

// The kernel; partials at `parts` (256-byte aligned, plan's bytes). p_out: the
// kernel's parameters for a merge.
struct PromptParams;
pa_status launch_prompt(const PromptCall& c, const PromptPlan& plan, void* parts, PromptParams* p_out);

}  // namespace pa
