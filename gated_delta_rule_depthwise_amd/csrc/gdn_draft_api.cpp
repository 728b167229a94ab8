// gdn_draft_api.cpp -- the C ABI's steps on drafted tokens: host-side validation and launches
// of gdn_draft, gdn_fold and gdn_verify. Every check runs before anything is enqueued.
#include <stdint.h>

#include "gdn.h"
#include "gdn_draft.h"

namespace {

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

int elem_bytes(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

int32_t qk_heads(const gdn_params *p) { return p->Hqk ? p->Hqk : p->H; }

// what gdn_draft and gdn_fold share: the configurations of a decode step, and a tape
int check_tape(const gdn_params *p, int kda, const gdn_tape *t, int32_t B, int32_t share)
{
    // the parameters' own check, as every entry point makes it (no plan is made of it)
    const int rc = gdn_segments(p, GDN_KIND_VARLEN | (kda ? GDN_PLAN_KDA : 0), 1, 1, 0);
    if (rc < 0)
        return rc;
    if (!((p->dk == 64 || p->dk == 128) && (p->dv == p->dk || p->dv == 2 * p->dk)))
        return GDN_E_UNSUPPORTED;
    // the grids (up to 4 workgroups of 256 threads per stream and head) stay below 2^32 threads
    if (B < 1 || share < 1 || B % share || (int64_t)B * p->H > (1 << 22))
        return GDN_E_ARG;
    if (!t || !t->k || !t->d || !t->g || !t->len || t->cap < 1 ||
        (p->conv_k > 0) != (t->raw != nullptr))
        return GDN_E_ARG;
    if (!aligned16(t->k) || !aligned16(t->d) || !aligned16(t->raw) ||
        (kda && !aligned16(t->g)))
        return GDN_E_ARG;
    return GDN_OK;
}

gdn::Tape device_tape(const gdn_tape *t)
{
    return gdn::Tape{t->k, t->d, t->g, t->raw, t->len, t->cap, t->status};
}

int draft(const gdn_params *p, int kda, const void *q, const void *k, const void *v,
          const float *g, const float *beta, const float *const *h_ptrs,
          const void *const *conv_state_ptrs, const float *conv_w, const gdn_tape *tape,
          void *o, int32_t B, int32_t T, int32_t share, void *stream)
{
    const int rc = check_tape(p, kda, tape, B, share);
    if (rc != GDN_OK)
        return rc;
    if (T < 1 || T > GDN_DRAFT_MAX_T || T > tape->cap)
        return GDN_E_ARG;
    if (!q || !k || !v || !g || !beta || !h_ptrs || !o)
        return GDN_E_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (kda && !aligned16(g)))
        return GDN_E_ARG;
    const bool front = p->conv_k > 0;
    if (front != (conv_w != nullptr) || front != (conv_state_ptrs != nullptr))
        return GDN_E_ARG;
    gdn::DraftArgs a{};
    a.q = q, a.k = k, a.v = v, a.ld = p->ld_qkv;
    a.g = g, a.beta = beta, a.h_ptrs = h_ptrs;
    a.conv_state_ptrs = conv_state_ptrs, a.conv_w = conv_w;
    a.tape = device_tape(tape);
    a.o = (float *)o;
    a.B = B, a.T = T, a.share = share;
    a.H = p->H, a.Hqk = qk_heads(p), a.dk = p->dk, a.dv = p->dv, a.K = p->conv_k;
    a.do_l2 = p->eps >= 0.f;
    a.eps = p->eps;
    a.scale = p->scale;
    a.z = p->z;
    a.ld_z = p->ld_z;
    a.norm_w = p->norm_w;
    a.norm_eps = p->norm_eps;
    return gdn::launch_draft(p->dtype, kda, a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_E_HIP;
}

int fold(const gdn_params *p, int kda, const float *const *h_ptrs,
         const void *const *conv_state_ptrs, float *const *h_out_ptrs,
         void *const *conv_out_ptrs, const gdn_tape *tape, int32_t *len_out, int32_t B,
         int32_t share, int32_t min_len, void *stream)
{
    const int rc = check_tape(p, kda, tape, B, share);
    if (rc != GDN_OK)
        return rc;
    if (!h_ptrs || !h_out_ptrs || min_len < 0)
        return GDN_E_ARG;
    const bool front = p->conv_k > 0;
    if (front != (conv_state_ptrs != nullptr) || front != (conv_out_ptrs != nullptr))
        return GDN_E_ARG;
    if (share > 1 && ((const void *)h_ptrs == (const void *)h_out_ptrs ||
                      (front && (const void *)conv_state_ptrs == (const void *)conv_out_ptrs)))
        return GDN_E_ARG;  // the streams of a state have states of their own after it
    gdn::FoldArgs a{};
    a.h_ptrs = h_ptrs, a.conv_state_ptrs = conv_state_ptrs;
    a.h_out_ptrs = h_out_ptrs, a.conv_out_ptrs = conv_out_ptrs;
    a.tape = device_tape(tape);
    a.len_out = len_out;
    a.B = B, a.share = share, a.min_len = min_len;
    a.H = p->H, a.Hqk = qk_heads(p), a.dk = p->dk, a.dv = p->dv, a.K = p->conv_k;
    return gdn::launch_fold(p->dtype, kda, a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_E_HIP;
}

// The parts a row of weights is cut into: multiples of 8192 elements (four rounds of loads
// of a workgroup's 4 waves) and at most 64 of them.
constexpr int32_t kVerifySeg = 8192, kVerifyParts = 64, kVerifyMaxT = 1024, kVerifyMaxV = 1 << 30,
                  kVerifyMaxB = 1 << 18;

bool verify_shape(int32_t B, int32_t T, int32_t V, int32_t *nseg, int32_t *seg)
{
    if (B < 1 || T < 0 || T > kVerifyMaxT || V < 1 || V > kVerifyMaxV || B > kVerifyMaxB)
        return false;
    int64_t s = ((int64_t)V + kVerifyParts - 1) / kVerifyParts;
    s = (s + kVerifySeg - 1) / kVerifySeg * kVerifySeg;
    *seg = (int32_t)s;
    *nseg = (int32_t)(((int64_t)V + s - 1) / s);
    return true;
}
}  // namespace

extern "C" {

int gdn_draft(const gdn_params *p, const void *q, const void *k, const void *v,
              const float *g, const float *beta, const float *const *h_ptrs,
              const void *const *conv_state_ptrs, const float *conv_w, const gdn_tape *tape,
              void *o, int32_t B, int32_t T, int32_t share, void *stream)
{
    return draft(p, 0, q, k, v, g, beta, h_ptrs, conv_state_ptrs, conv_w, tape, o, B, T, share,
                 stream);
}

int kda_draft(const gdn_params *p, const void *q, const void *k, const void *v,
              const float *g, const float *beta, const float *const *h_ptrs,
              const void *const *conv_state_ptrs, const float *conv_w, const gdn_tape *tape,
              void *o, int32_t B, int32_t T, int32_t share, void *stream)
{
    return draft(p, 1, q, k, v, g, beta, h_ptrs, conv_state_ptrs, conv_w, tape, o, B, T, share,
                 stream);
}

int gdn_fold(const gdn_params *p, const float *const *h_ptrs,
             const void *const *conv_state_ptrs, float *const *h_out_ptrs,
             void *const *conv_out_ptrs, const gdn_tape *tape, int32_t *len_out, int32_t B,
             int32_t share, int32_t min_len, void *stream)
{
    return fold(p, 0, h_ptrs, conv_state_ptrs, h_out_ptrs, conv_out_ptrs, tape, len_out, B,
                share, min_len, stream);
}

int kda_fold(const gdn_params *p, const float *const *h_ptrs,
             const void *const *conv_state_ptrs, float *const *h_out_ptrs,
             void *const *conv_out_ptrs, const gdn_tape *tape, int32_t *len_out, int32_t B,
             int32_t share, int32_t min_len, void *stream)
{
    return fold(p, 1, h_ptrs, conv_state_ptrs, h_out_ptrs, conv_out_ptrs, tape, len_out, B,
                share, min_len, stream);
}

size_t gdn_verify_workspace_bytes(int32_t B, int32_t T, int32_t V)
{
    int32_t nseg = 0, seg = 0;
    if (!verify_shape(B, T, V, &nseg, &seg))
        return 0;
    return align_up((size_t)B * nseg * sizeof(double)) + align_up((size_t)B * 2 * sizeof(int32_t));
}

int gdn_verify(const void *target, int64_t ld_target, const void *draft_p, int64_t ld_draft,
               int32_t dtype, const int32_t *tokens, const int32_t *num_drafts,
               const float *u, int32_t B, int32_t T, int32_t V, int32_t *accepted,
               int32_t *next, int32_t *len, void *ws, size_t ws_bytes, void *stream)
{
    gdn::VerifyArgs a{};
    if (!verify_shape(B, T, V, &a.nseg, &a.seg))
        return GDN_E_ARG;
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return GDN_E_UNSUPPORTED;
    if (!target || !u || !accepted || !next || (T > 0 && !tokens) || ld_target < V ||
        (draft_p && ld_draft < V))
        return GDN_E_ARG;
    const uintptr_t em = (uintptr_t)elem_bytes(dtype) - 1;
    if (((uintptr_t)target & em) || ((uintptr_t)draft_p & em))
        return GDN_E_ARG;
    if (ws_bytes < gdn_verify_workspace_bytes(B, T, V) || !ws)
        return GDN_E_WORKSPACE;
    if (!aligned16(ws))
        return GDN_E_ARG;
    a.target = target, a.draft = draft_p, a.ld_target = ld_target, a.ld_draft = ld_draft;
    a.tokens = tokens, a.num_drafts = num_drafts, a.u = u;
    a.B = B, a.T = T, a.V = V;
    a.accepted = accepted, a.next = next, a.len = len;
    a.part = (double *)ws;
    a.info = (int32_t *)((char *)ws + align_up((size_t)B * a.nseg * sizeof(double)));
    return gdn::launch_verify(dtype, a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_E_HIP;
}

}  // extern "C"
