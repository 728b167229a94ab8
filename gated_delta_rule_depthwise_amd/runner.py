"""Device buffers for one workload and the C-ABI call that processes them.

Plumbing only: torch allocates device memory and provides the stream; every step of the
path runs inside libgdn's kernels (binding.py). Used by the tests and by bench.py.
"""
from __future__ import annotations

import torch

from . import binding as B


class Prefill:
    """One call of gdn_prefill / kda_prefill / gdn_prefill_batched / gdn_prefill_varlen.

    ``inp`` is a dict from :func:`inputs.make`. ``mode`` is "single", "batched" or
    "varlen" (default: single for one stream, batched for equal lengths, else varlen).
    ``o_fill`` pre-fills the output so rows the call must not write can be checked.
    ``segmented=False`` gives the call a workspace without room for segment states.
    """

    def __init__(self, inp: dict, device="cuda", mode=None, o_fill=0.0, eps=None,
                 scale=None, segmented=True):
        spec = inp["spec"]
        self.spec = spec
        self.device = device
        lens = list(spec.lengths)
        if mode is None:
            mode = "single" if len(lens) == 1 else (
                "batched" if len(set(lens)) == 1 else "varlen")
        self.mode = mode
        self.x = inp["x"].to(device)
        self.g = inp["g"].to(device)
        self.beta = inp["beta"].to(device)
        self.h0 = inp["h0"].to(device)
        self.h = self.h0.clone()
        self.cu = inp["cu_seqlens"].to(device)
        self.conv_w = None if inp["conv_w"] is None else inp["conv_w"].to(device)
        self.conv_state0 = None if inp["conv_state"] is None else inp["conv_state"].to(device)
        self.conv_state = None if self.conv_state0 is None else self.conv_state0.clone()
        self.o = torch.full((spec.alloc, spec.H, spec.dv), o_fill, dtype=torch.float32,
                            device=device)
        self.h_ptrs = torch.tensor([self.h[b].data_ptr() for b in range(spec.B)],
                                   dtype=torch.int64, device=device)
        self.cs_ptrs = None if self.conv_state is None else torch.tensor(
            [self.conv_state[b].data_ptr() for b in range(spec.B)], dtype=torch.int64,
            device=device)
        self.z = None if inp.get("z") is None else inp["z"].to(device)
        self.norm_w = None if inp.get("norm_w") is None else inp["norm_w"].to(device)
        self.params = B.params(
            spec.H, spec.dk, spec.dv, chunk=spec.chunk,
            eps=spec.eps if eps is None else eps,
            scale=spec.scale if scale is None else scale,
            dtype=B.GDN_BF16 if spec.dtype == "bf16" else B.GDN_F32,
            conv_k=spec.conv_k if spec.front_end else 0, ld_qkv=spec.cd,
            z=self.z, norm_w=self.norm_w, norm_eps=spec.norm_eps, Hqk=spec.Hqk)
        kind = {"single": B.GDN_KIND_SINGLE, "batched": B.GDN_KIND_BATCHED,
                "varlen": B.GDN_KIND_VARLEN}[mode]
        self.kind = kind
        # the kind to ask gdn_segments / gdn_segment_plan with: the plan of this call's gate
        self.plan_kind = kind | (B.GDN_PLAN_KDA if spec.gate == "kda" else 0)
        # segmented=False sizes the workspace for the front end only, which makes a single
        # or batched call run its scan unsegmented
        self.ws_bytes = B.gdn_workspace_bytes(
            self.params, spec.B, spec.N,
            (kind if segmented else B.GDN_KIND_VARLEN) | (self.plan_kind & B.GDN_PLAN_KDA))
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=device)
        es = self.x.element_size()
        base = self.x.data_ptr()
        self.q_ptr = base
        self.k_ptr = base + spec.qk_heads * spec.dk * es
        self.v_ptr = base + 2 * spec.qk_heads * spec.dk * es

    def reset(self):
        """Restore the initial states (h, conv window)."""
        self.h.copy_(self.h0)
        if self.conv_state is not None:
            self.conv_state.copy_(self.conv_state0)

    def __call__(self, stream=None) -> int:
        s = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        sp = self.spec
        cs = None if self.conv_state is None else self.conv_state
        if self.mode == "single":
            fn = B.kda_prefill if sp.gate == "kda" else B.gdn_prefill
            return fn(self.params, self.q_ptr, self.k_ptr, self.v_ptr, self.g, self.beta,
                      self.h, cs, self.conv_w, self.o, sp.N, self.ws, self.ws_bytes, s)
        kda = sp.gate == "kda"
        if self.mode == "batched":
            fn = B.kda_prefill_batched if kda else B.gdn_prefill_batched
            return fn(self.params, self.q_ptr, self.k_ptr, self.v_ptr, self.g, self.beta,
                      self.h_ptrs, self.cs_ptrs, self.conv_w, self.o, sp.B, sp.lengths[0],
                      self.ws, self.ws_bytes, s)
        fn = B.kda_prefill_varlen if kda else B.gdn_prefill_varlen
        return fn(self.params, self.q_ptr, self.k_ptr, self.v_ptr, self.g, self.beta,
                  self.h_ptrs, self.cs_ptrs, self.conv_w, self.o, self.cu, sp.B, sp.N,
                  max(sp.lengths), self.ws, self.ws_bytes, s)


class Decode:
    """One call of gdn_decode / kda_decode: row b of ``inp`` is stream b's new token.

    ``inp`` is a dict from :func:`inputs.make` whose streams all have length 1. The states
    h (``[B, H, dk, dv]``) and the conv windows are updated in place by every call; ``o`` is
    ``[B, H, dv]``. ``step(t, ...)`` points the call at other token rows (see there).
    """

    def __init__(self, inp: dict, device="cuda", o_fill=0.0, eps=None, scale=None):
        spec = inp["spec"]
        self.spec = spec
        self.device = device
        self.x = inp["x"].to(device)
        self.g = inp["g"].to(device)
        self.beta = inp["beta"].to(device)
        self.h0 = inp["h0"].to(device)
        self.h = self.h0.clone()
        self.conv_w = None if inp["conv_w"] is None else inp["conv_w"].to(device)
        self.conv_state0 = None if inp["conv_state"] is None else inp["conv_state"].to(device)
        self.conv_state = None if self.conv_state0 is None else self.conv_state0.clone()
        self.o = torch.full((spec.B, spec.H, spec.dv), o_fill, dtype=torch.float32,
                            device=device)
        self.h_ptrs = torch.tensor([self.h[b].data_ptr() for b in range(spec.B)],
                                   dtype=torch.int64, device=device)
        self.cs_ptrs = None if self.conv_state is None else torch.tensor(
            [self.conv_state[b].data_ptr() for b in range(spec.B)], dtype=torch.int64,
            device=device)
        self.eps = spec.eps if eps is None else eps
        self.scale = spec.scale if scale is None else scale
        self.z = None if inp.get("z") is None else inp["z"].to(device)
        self.norm_w = None if inp.get("norm_w") is None else inp["norm_w"].to(device)
        self.params = self._params(spec.cd)
        es = self.x.element_size()
        base = self.x.data_ptr()
        self.q_ptr = base
        self.k_ptr = base + spec.qk_heads * spec.dk * es
        self.v_ptr = base + 2 * spec.qk_heads * spec.dk * es

    def _params(self, ld, z=None, ld_z=None):
        sp = self.spec
        return B.params(sp.H, sp.dk, sp.dv, chunk=sp.chunk, eps=self.eps, scale=self.scale,
                        dtype=B.GDN_BF16 if sp.dtype == "bf16" else B.GDN_F32,
                        conv_k=sp.conv_k if sp.front_end else 0, ld_qkv=ld,
                        z=self.z if z is None else z, norm_w=self.norm_w, ld_z=ld_z,
                        norm_eps=sp.norm_eps, Hqk=sp.Hqk)

    def reset(self):
        """Restore the initial states (h, conv window)."""
        self.h.copy_(self.h0)
        if self.conv_state is not None:
            self.conv_state.copy_(self.conv_state0)

    def _call(self, p, q, k, v, g, beta, stream):
        s = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        fn = B.kda_decode if self.spec.gate == "kda" else B.gdn_decode
        return fn(p, q, k, v, g, beta, self.h_ptrs, self.cs_ptrs, self.conv_w, self.o,
                  self.spec.B, s)

    def __call__(self, stream=None) -> int:
        return self._call(self.params, self.q_ptr, self.k_ptr, self.v_ptr, self.g,
                          self.beta, stream)

    def step(self, x, t, T, g, beta, stream=None) -> int:
        """Decode token t of T per stream from prefill-layout rows: stream b's token is row
        b*T + t of ``x`` (a device tensor of packed rows; the row stride between streams
        is T rows); ``g`` and ``beta`` hold this step's [B, H(, dk)] values. With the
        output gate, ``self.z`` must hold the T rows per stream in the same layout."""
        sp = self.spec
        es = x.element_size()
        base = x.data_ptr() + t * sp.cd * es
        # the output gate's z in the same prefill layout: stream b's row b*T + t
        zp = None if self.z is None else self.z.data_ptr() + t * sp.H * sp.dv * es
        p = self._params(T * sp.cd, zp, T * sp.H * sp.dv)
        return self._call(p, base, base + sp.qk_heads * sp.dk * es,
                          base + 2 * sp.qk_heads * sp.dk * es, g, beta, stream)


class Drafts:
    """Streams with tapes: gdn_draft / kda_draft and gdn_fold / kda_fold on one set of device
    buffers.

    ``spec`` is an :class:`inputs.Spec` (its heads, dims, dtype, gate, conv and output gate; the
    lengths are not used). ``share`` consecutive streams read one state. ``h`` is
    ``[B/share, H, dk, dv]``, ``conv_state`` ``[B/share, cd, K-1]``; the tapes hold ``cap``
    entries per stream (``k``, ``d``, ``g``, ``raw``) and start empty (``len`` zero).
    """

    def __init__(self, spec, B_, cap, h, conv_state=None, conv_w=None, share=1, device="cuda",
                 norm_w=None, fill=0.0, eps=None, scale=None):
        self.spec, self.B, self.cap, self.share, self.device = spec, B_, cap, share, device
        td = spec.torch_dtype
        self.eps = spec.eps if eps is None else eps
        self.scale = spec.scale if scale is None else scale
        self.h = h.to(device)
        self.conv_state = None if conv_state is None else conv_state.to(device)
        self.conv_w = None if conv_w is None else conv_w.to(device)
        self.norm_w = None if norm_w is None else norm_w.to(device)
        gw = (spec.dk,) if spec.gate == "kda" else ()
        f32 = dict(dtype=torch.float32, device=device)
        self.k = torch.full((B_, cap, spec.qk_heads, spec.dk), fill, **f32)
        self.d = torch.full((B_, cap, spec.H, spec.dv), fill, **f32)
        self.g = torch.full((B_, cap, spec.H) + gw, fill, **f32)
        self.raw = None if self.conv_w is None else torch.full(
            (B_, cap, spec.cd), fill, dtype=td, device=device)
        self.len = torch.zeros(B_, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.h_ptrs = self._ptrs(self.h)
        self.cs_ptrs = None if self.conv_state is None else self._ptrs(self.conv_state)

    def _ptrs(self, t):
        return torch.tensor([t[i].data_ptr() for i in range(t.shape[0])], dtype=torch.int64,
                            device=self.device)

    def tape(self):
        return B.tape(self.k, self.d, self.g, self.raw, self.len, self.cap, self.status)

    def params(self, ld=None, z=None, ld_z=None):
        sp = self.spec
        return B.params(sp.H, sp.dk, sp.dv, eps=self.eps, scale=self.scale,
                        dtype=B.GDN_BF16 if sp.dtype == "bf16" else B.GDN_F32,
                        conv_k=0 if self.conv_w is None else sp.conv_k,
                        ld_qkv=sp.cd if ld is None else ld, z=z,
                        norm_w=None if z is None else self.norm_w, ld_z=ld_z,
                        norm_eps=sp.norm_eps, Hqk=sp.Hqk)

    def draft(self, x, g, beta, o, T, z=None, stream=None) -> int:
        """T tokens per stream from rows ``x`` [B*T, >= cd] (row stride = its own), gates and
        betas, into ``o`` [B*T, H, dv]."""
        sp = self.spec
        s = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        es, base = x.element_size(), x.data_ptr()
        p = self.params(x.stride(0), z, None if z is None else z.stride(0))
        fn = B.kda_draft if sp.gate == "kda" else B.gdn_draft
        return fn(p, base, base + sp.qk_heads * sp.dk * es, base + 2 * sp.qk_heads * sp.dk * es,
                  g, beta, self.h_ptrs, self.cs_ptrs, self.conv_w, self.tape(), o, self.B, T,
                  self.share, s)

    def fold(self, h_out=None, conv_out=None, len_out=None, min_len=0, stream=None) -> int:
        """Fold into ``h_out`` / ``conv_out`` (None: in place, share 1); ``len_out`` None:
        the tapes' own lengths are cleared."""
        s = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        hp = self.h_ptrs if h_out is None else self._ptrs(h_out)
        cp = self.cs_ptrs if conv_out is None else self._ptrs(conv_out)
        self._kept = (hp, cp)  # the call reads them after it returns
        fn = B.kda_fold if self.spec.gate == "kda" else B.gdn_fold
        return fn(self.params(), self.h_ptrs, self.cs_ptrs, hp, cp, self.tape(),
                  self.len if len_out is None else len_out, self.B, self.share, min_len, s)


def verify(target, tokens, u, draft=None, num=None, len=None, stream=None):
    """gdn_verify on device tensors: target [B, T+1, V], draft [B, T, V] or None, tokens
    [B, T] int32, u [B, T+1]. Returns (status, accepted [B], next [B])."""
    Bn, T1, V = target.shape
    dev = target.device
    s = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
    n = B.gdn_verify_workspace_bytes(Bn, T1 - 1, V)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    acc = torch.full((Bn,), -7, dtype=torch.int32, device=dev)
    nxt = torch.full((Bn,), -7, dtype=torch.int32, device=dev)
    rc = B.gdn_verify(target, target.stride(1), draft, V if draft is None else draft.stride(1),
                      B.GDN_BF16 if target.dtype == torch.bfloat16 else B.GDN_F32, tokens, num, u,
                      Bn, T1 - 1, V, acc, nxt, len, ws, n, s)
    return rc, acc, nxt
