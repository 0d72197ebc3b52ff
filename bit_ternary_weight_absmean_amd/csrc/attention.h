// Arguments and plans of the attention kernels, shared by the ABI and csrc/attention.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bt {

struct AttnArgs {
    const void *q, *k, *v;
    const int *q_start, *k_start, *k_len;
    void *out;
    float *lse;
    float *ws_o, *ws_l;  // slices' outputs and lse (ws_o: the whole workspace for launch_attention)
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;  // strides in elements
    int T, S, B, P;
    int Hq, Hkv, G, D;
    float scale_log2;  // scale * log2(e)
    int causal;
    int target, min_units;  // items per key head to cut the keys into (0: no cut), smallest slice
    int items;              // items per key head that the launch has
    int shared;             // k, v are the shared prefix of all T tokens
    int pieced;             // every item goes to the workspace
};

// One launch's work items: row tiles of bm rows, at most `items` items per key head.
struct AttnPart {
    int bm, min_units;
    int64_t tiles, target, items;
    int64_t o_off, l_off;  // in the workspace
};

struct AttnPlan {
    AttnPart main, pre;
    size_t bytes;
};

AttnPlan attn_plan(int64_t T, int64_t S, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t P);
hipError_t launch_attention(const AttnArgs &args, const AttnArgs &prefix, const AttnPlan &p, int type, int out_type,
                            hipStream_t s);

}  // namespace bt
