// gdn_draft.h -- argument blocks of the steps on drafted tokens (gdn_draft_api.cpp to
// gdn_draft.hip and gdn_verify.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

// The streams' tapes: tokens appended to a state that is left as it is (see gdn.h).
struct Tape {
    float *k;      // [B][cap][Hqk][dk]
    float *d;      // [B][cap][H][dv]
    float *g;      // [B][cap][H] or [B][cap][H][dk]
    void *raw;     // [B][cap][cd] (K > 0)
    int32_t *len;  // [B]
    int32_t cap;
    int32_t *status;  // nullptr, or ORed with GDN_BAD_TAPE for a length out of range
};

// T tokens per stream against states that are only read, and the tapes' new entries.
struct DraftArgs {
    const void *q, *k, *v;           // row b*T + t: q + row*ld + h*dk, ...
    int64_t ld;
    const float *g;                  // [B*T][H] or [B*T][H][dk]
    const float *beta;               // [B*T][H]
    const float *const *h_ptrs;      // [B/share], each [H][dk][dv]
    const void *const *conv_state_ptrs;  // [B/share], each [cd][K-1] (K > 0)
    const float *conv_w;             // [cd][K] (K > 0)
    Tape tape;
    float *o;                        // [B*T][H][dv]
    int32_t B, T, share, H, Hqk, dk, dv, K;
    int32_t do_l2;
    float eps, scale;
    const void *z;                   // output gate (nullptr: off): row r at z + r*ld_z
    int64_t ld_z;
    const float *norm_w;             // [dv]
    float norm_eps;
};

// The tapes worked into the states.
struct FoldArgs {
    const float *const *h_ptrs;          // [B/share]
    const void *const *conv_state_ptrs;  // [B/share] (K > 0)
    float *const *h_out_ptrs;            // [B]
    void *const *conv_out_ptrs;          // [B] (K > 0)
    Tape tape;
    int32_t *len_out;                    // [B], or nullptr; tape.len itself: cleared after
    int32_t B, share, min_len, H, Hqk, dk, dv, K;
};

// Drafted tokens against the target's probabilities. A row of V weights is cut into nseg
// parts of seg elements for the sums.
struct VerifyArgs {
    const void *target, *draft;      // rows b*(T+1)+t and b*T+t; draft nullptr: one-hot
    int64_t ld_target, ld_draft;
    const int32_t *tokens, *num_drafts;
    const float *u;
    int32_t B, T, V;
    int32_t *accepted, *next, *len;
    double *part;                    // [B][nseg]: sums of the weights
    int32_t *info;                   // [B][2]: drafts accepted, drafts
    int32_t nseg, seg;
};

// Return hipSuccess or the launch error.
hipError_t launch_draft(int dtype, int kda, const DraftArgs &a, hipStream_t s);
hipError_t launch_fold(int dtype, int kda, const FoldArgs &a, hipStream_t s);
hipError_t launch_verify(int dtype, const VerifyArgs &a, hipStream_t s);

}  // namespace gdn
