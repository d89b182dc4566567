// What the kernels of decode_runs.cu and decode_runs_tc.cu share.
#pragma once

#include "kernels.h"
#include "vec.cuh"

namespace gdn {

constexpr int kRunTokens = 8;  // tokens taken at once

// The decay and the write strength of a token as the recurrence uses them; with logits
// alpha = exp(-softplus(x)) = 1 / (1 + e^x).
__device__ __forceinline__ float2 decay_pair(float la, float be, unsigned flags) {
    if (flags & kFlagGateLogits) return make_float2(sigmoid(-la), sigmoid(be));
    return make_float2(expf(la), be);
}

// Whether an earlier sequence with tokens names this slot (seen by every lane that
// calls with its own share of the sequences).
__device__ __forceinline__ int slot_taken(const RunsArgs &a, int n, int slot, int from, int step) {
    int taken = 0;
    for (int i = from; i < n; i += step)
        if (a.slots[i] == slot) taken |= !a.cu || a.cu[i] < a.cu[i + 1];
    return taken;
}

}  // namespace gdn
