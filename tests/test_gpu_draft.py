"""gdn_draft / kda_draft and gdn_fold / kda_fold against their definition in float64.

Tolerance: both run in fp32 throughout. An output is a sum of dk products with the state plus
one per tape entry and new token, each factor off by a few roundings (conv, SiLU, L2, gates):
N = dk + n + T + 32 steps of at most 2^-24 relative to the sum of the terms' magnitudes. That
sum is at most sqrt(dk) times the RMS of the terms' own sum for terms of random sign, and an
element's share of it up to about 5 times that at these sizes (d = 128, n up to 70):
250 * 6e-8 * 11 * 5 / 8 = 1e-4 of the outputs' RMS, the bar of the decode step. The keys are a
conv of 4 products, a SiLU and a division by a norm of 128 squares (a tree over 16 lanes of 8):
(4 + 8 + 8 + 4) * 6e-8 < 2e-6 of an element of RMS 1/sqrt(dk), at most 10 times its RMS: 2e-5.
Windows, raw rows, log-gates and everything a call must not touch are compared bit for bit."""
import dataclasses

import numpy as np
import pytest
import torch

from gated_delta_rule_depthwise_amd import binding as G
from gated_delta_rule_depthwise_amd import inputs
from gated_delta_rule_depthwise_amd.runner import Decode, Drafts, verify
from tests import draft_ref
from tests.gpu_util import rel_err

pytestmark = pytest.mark.gpu

TOL, TOL_K, SENT = 1e-4, 2e-5, -12345.0


def spec_of(H=2, Hqk=0, dk=128, dv=128, dtype="bf16", gate="gdn", conv_k=4, z=False):
    s = dataclasses.replace(inputs.decode_config(1), H=H, Hqk=Hqk, dk=dk, dv=dv, dtype=dtype, gate=gate,
                            out_gate=z, conv_k=conv_k or 4, front_end=conv_k > 0)
    return s


def make(spec, B, cap, lens, share=1, seed=0, dist="uniform", fill=float("nan"), **kw):
    """Streams with random states, windows and tapes of the given lengths; entries past a
    tape's end hold ``fill``."""
    r = np.random.default_rng(seed)
    td = spec.torch_dtype
    P = B // share

    def normal(*s, std=1.0):
        return torch.from_numpy((r.standard_normal(s) * std).astype(np.float32))

    conv = spec.front_end
    st = Drafts(spec, B, cap, normal(P, spec.H, spec.dk, spec.dv, std=0.1),
                normal(P, spec.cd, spec.conv_k - 1).to(td) if conv else None,
                normal(spec.cd, spec.conv_k, std=0.5) if conv else None, share=share, fill=fill,
                norm_w=torch.from_numpy(r.uniform(0.5, 1.5, spec.dv).astype(np.float32)), **kw)
    for b, n in enumerate(lens):
        k = normal(n, spec.qk_heads, spec.dk)
        st.k[b, :n] = (k / k.norm(dim=-1, keepdim=True)).cuda()
        st.d[b, :n] = normal(n, spec.H, spec.dv, std=0.5).cuda()
        st.g[b, :n] = gates(r, dist, n, *st.g.shape[2:]).cuda()
        if conv:
            st.raw[b, :n] = normal(n, spec.cd).to(td).cuda()
    st.len.copy_(torch.tensor(lens, dtype=torch.int32))
    return st


def gates(r, dist, *shape):
    lo, hi = dict(uniform=(-0.5, -0.01), slow=(-0.02, -1e-4), strong=(-60.0, -5.0))[dist]
    return torch.from_numpy(r.uniform(lo, hi, shape).astype(np.float32))


def rows_of(spec, N, seed=1, dist="uniform", extra=0, z=False):
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((N, spec.cd + extra)).astype(np.float32)).to(spec.torch_dtype)
    gshape = (spec.H, spec.dk) if spec.gate == "kda" else (spec.H,)
    beta = torch.from_numpy((1 / (1 + np.exp(-r.standard_normal((N, spec.H))))).astype(np.float32))
    out = [x.cuda(), gates(r, dist, N, *gshape).cuda(), beta.cuda()]
    zz = torch.from_numpy(r.standard_normal((N, spec.H * spec.dv + extra)).astype(np.float32)).to(spec.torch_dtype)
    return out + [zz.cuda() if z else None]


def bits(t):
    return t.contiguous().view(torch.uint8)


def snapshot(st):
    return {n: getattr(st, n).clone() for n in ("h", "conv_state", "k", "d", "g", "raw", "len")
            if getattr(st, n) is not None}


def check_draft(st, x, g, beta, T, z=None, skip=()):
    """Runs the call and checks everything that it writes and must not write."""
    before = snapshot(st)
    lens = st.len.cpu().tolist()
    o = torch.full((st.B * T + 3, st.spec.H, st.spec.dv), SENT, device="cuda")
    assert st.draft(x, g, beta, o, T, z=z) == 0
    torch.cuda.synchronize()
    ok = [b for b in range(st.B) if b not in skip]
    for b in skip:                                    # the reference walks valid lengths only
        st.len[b] = 0
    after = {n: t.clone() for n, t in snapshot(st).items()}
    for n, t in before.items():                       # the reference works on the tapes as they were
        getattr(st, n).copy_(t)
    for b in skip:
        st.len[b] = 0
    zref = None if z is None else z[:, :st.spec.H * st.spec.dv]
    ro, rk, rd = draft_ref.draft(st, x, g, beta, T, z=zref)
    sel = [b * T + t for b in ok for t in range(T)]
    if z is None:
        assert rel_err(o[sel].cpu().numpy(), ro[sel]) <= TOL
    else:  # the gate divides rows by their own RMS: rows compare at their own scale
        got, ref = o[sel].cpu().numpy().astype(np.float64), ro[sel]
        assert np.abs(got - ref).max() <= TOL * 10 * np.abs(ref).max()
    assert bool((o[st.B * T:] == SENT).all()), "o written past the last row"
    for b in skip:
        assert bool((o[b * T:(b + 1) * T] == SENT).all()), "o of a stream that is left out"
    want = {n: t.clone() for n, t in before.items()}
    for b in ok:
        n = lens[b]
        assert rel_err(after["k"][b, n:n + T].cpu().numpy(), rk[b]) <= TOL_K
        assert rel_err(after["d"][b, n:n + T].cpu().numpy(), rd[b]) <= TOL
        want["k"][b, n:n + T], want["d"][b, n:n + T] = after["k"][b, n:n + T], after["d"][b, n:n + T]
        want["g"][b, n:n + T] = g[b * T:(b + 1) * T]
        if "raw" in want:
            want["raw"][b, n:n + T] = x[b * T:(b + 1) * T, :st.spec.cd]
    for n, t in want.items():
        if n != "len":
            assert torch.equal(bits(after[n]), bits(t)), "%s: written where it must not be" % n
            getattr(st, n).copy_(after[n])
    st.len.copy_(torch.tensor(lens, dtype=torch.int32))
    return o[:st.B * T]


CASES = {
    "one token, empty tape": dict(B=1, T=1, lens=[0]),
    "one token, odd heads": dict(B=3, T=1, H=3, lens=[0, 1, 2], cap=3),
    "16 tokens": dict(B=2, T=16, lens=[0, 19], cap=35),
    "9 tokens": dict(B=2, T=9, lens=[3, 16], cap=25),
    "8 tokens, no conv": dict(B=3, T=8, conv_k=0, lens=[0, 15, 17], cap=25),
    "tapes around a block": dict(B=7, T=2, H=1, lens=[14, 15, 16, 17, 31, 32, 33], cap=35),
    "long tape, slow gates": dict(B=2, T=3, H=1, lens=[70, 64], cap=80, dist="slow"),
    "strong gates": dict(B=2, T=4, H=1, lens=[20, 5], cap=30, dist="strong"),
    "conv of 2": dict(B=3, T=2, conv_k=2, lens=[0, 1, 2], cap=4),
    "conv of 3": dict(B=4, T=3, conv_k=3, lens=[0, 1, 2, 3], cap=6),
    "shared q/k heads": dict(B=3, T=5, H=6, Hqk=2, lens=[0, 4, 9], cap=16),
    "shared prefix": dict(B=22, T=3, H=2, share=11, lens=list(range(22)), cap=26),
    "shared prefix, one token": dict(B=17, T=1, H=1, share=17, lens=[i % 5 for i in range(17)], cap=8),
    "shared prefix, 16 tokens": dict(B=3, T=16, H=1, share=3, lens=[0, 7, 18], cap=34),
    "wide values": dict(B=2, T=3, H=2, dv=256, lens=[0, 18], cap=22),
    "wide values, 16 tokens": dict(B=1, T=16, H=1, dv=256, lens=[5], cap=24),
    "d 64": dict(B=3, T=4, H=2, dk=64, dv=64, lens=[0, 3, 20], cap=24),
    "f32 d 64": dict(B=3, T=4, H=2, dk=64, dv=64, dtype="f32", lens=[0, 3, 20], cap=24),
    "f32 64 x 128": dict(B=2, T=12, H=2, dk=64, dv=128, dtype="f32", conv_k=0, lens=[0, 17], cap=32),
    "kda": dict(B=3, T=3, gate="kda", lens=[0, 16, 21], cap=24),
    "kda 16 tokens": dict(B=2, T=16, H=1, gate="kda", lens=[2, 33], cap=50, dist="slow"),
    "kda strong": dict(B=2, T=5, H=1, gate="kda", lens=[9, 33], cap=50, dist="strong"),
    "kda shared": dict(B=18, T=2, H=4, Hqk=2, gate="kda", share=9, lens=[i for i in range(18)], cap=20),
    "kda wide": dict(B=1, T=16, H=1, dv=256, gate="kda", lens=[17], cap=40),
    "kda f32": dict(B=2, T=6, H=2, dk=64, dv=128, gate="kda", dtype="f32", conv_k=3, lens=[1, 16], cap=24),
    "output gate": dict(B=3, T=3, z=True, lens=[0, 5, 17], cap=24),
    "output gate, kda, d 64": dict(B=9, T=2, H=2, dk=64, dv=64, gate="kda", z=True, share=3,
                                   lens=[1] * 9, cap=4),
    "output gate, wide": dict(B=2, T=4, H=1, dv=256, z=True, lens=[0, 3], cap=8),
    "strided rows": dict(B=3, T=3, H=2, z=True, extra=24, lens=[0, 2, 4], cap=8),
}


def build(case, seed):
    case = dict(case)
    B, T, lens = case.pop("B"), case.pop("T"), case.pop("lens")
    cap, share = case.pop("cap", T), case.pop("share", 1)
    dist, extra = case.pop("dist", "uniform"), case.pop("extra", 0)
    spec = spec_of(**case)
    st = make(spec, B, cap, lens, share=share, seed=seed, dist=dist)
    return st, rows_of(spec, B * T, seed + 1, dist, extra, z=spec.out_gate), T


@pytest.mark.parametrize("name", CASES)
def test_draft_matches_definition(name):
    st, (x, g, beta, z), T = build(CASES[name], 5)
    check_draft(st, x, g, beta, T, z=z)


def test_draft_without_l2():
    spec = spec_of(H=2, dk=64, dv=64, dtype="f32", conv_k=0)
    st = make(spec, 2, 9, [0, 4], seed=2, eps=-1.0, scale=0.3)
    x, g, beta, _ = rows_of(spec, 8, 3)
    x = x * 0.125
    check_draft(st, x, g, beta, 4)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_bad_lengths_leave_a_stream_out(gate):
    """A tape length below 0, or without room for the tokens, leaves its stream alone; the
    other streams of the same state run, and the tape's status says so."""
    spec = spec_of(H=2, gate=gate)
    st = make(spec, 6, 8, [0, 3, 5, 2, 1, 5], share=3, seed=4)
    st.len[1], st.len[3], st.len[5] = -1, 6, 2147483647
    x, g, beta, _ = rows_of(spec, 18, 5)
    assert int(st.status) == 0
    check_draft(st, x, g, beta, 3, skip=(1, 3, 5))
    assert int(st.status) == G.GDN_BAD_TAPE
    st.status.zero_()
    h_out = torch.full((6,) + tuple(st.h.shape[1:]), SENT, device="cuda")
    c_out = torch.full((6,) + tuple(st.conv_state.shape[1:]), 3.0, dtype=torch.bfloat16, device="cuda")
    len_out = torch.full((6,), -9, dtype=torch.int32, device="cuda")
    assert st.fold(h_out, c_out, len_out) == 0
    assert int(st.status) == G.GDN_BAD_TAPE
    assert len_out.tolist() == [0, -1, 0, 0, 0, 2147483647]       # length 6 of 8 folds
    for b in (1, 5):
        assert bool((h_out[b] == SENT).all()) and bool((c_out[b] == 3.0).all())


@pytest.mark.parametrize("gate,share", [("gdn", 1), ("gdn", 4), ("kda", 4)])
def test_nan_reaches_nothing_else(gate, share):
    """NaN in one stream's tape, in one stream's rows and in the rows after a token: the other
    streams (of the same state too) and the tokens before it come out bit for bit the same."""
    spec = spec_of(H=2, gate=gate, conv_k=4)
    st = make(spec, 4, 24, [17, 4, 0, 9], share=share, seed=6, fill=0.0)
    x, g, beta, _ = rows_of(spec, 12, 7)
    o = torch.empty(12, 2, 128, device="cuda")
    assert st.draft(x, g, beta, o, 3) == 0
    torch.cuda.synchronize()
    want, tapes = o.clone(), snapshot(st)
    for b in range(4):
        st.k[b, int(st.len[b]):], st.d[b, int(st.len[b]):], st.g[b, int(st.len[b]):] = (float("nan"),) * 3
    st.d[0, 5], st.k[1, 2], st.raw[1, 3] = float("inf"), float("nan"), float("nan")
    x[2 * 3 + 1:2 * 3 + 3] = float("nan")                        # tokens 1, 2 of stream 2
    g[3 * 3 + 2], beta[3 * 3 + 2] = float("nan"), float("nan")   # token 2 of stream 3
    assert st.draft(x, g, beta, o, 3) == 0
    torch.cuda.synchronize()
    for r in (6, 9, 10):
        assert torch.equal(o[r], want[r]), r
    assert torch.equal(st.d[2, 0], tapes["d"][2, 0]) and torch.equal(st.d[3, 9:11], tapes["d"][3, 9:11])
    assert not bool(torch.isfinite(o[0:6]).any())


FOLDS = {
    "in place": dict(B=3, lens=[0, 5, 17], cap=20),
    "one entry": dict(B=2, lens=[1, 1], cap=1, H=3),
    "around a block": dict(B=6, H=1, lens=[15, 16, 17, 31, 32, 33], cap=33),
    "long": dict(B=2, H=1, lens=[100, 64], cap=100, dist="slow"),
    "shared": dict(B=6, share=3, lens=[0, 1, 2, 3, 4, 5], cap=8, H=4, Hqk=2),
    "conv of 2": dict(B=3, lens=[0, 1, 2], cap=3, conv_k=2),
    "no conv": dict(B=3, lens=[0, 1, 9], cap=9, conv_k=0),
    "d 64": dict(B=3, dk=64, dv=64, lens=[3, 20, 0], cap=24),
    "wide": dict(B=2, dv=256, lens=[3, 20], cap=24),
    "f32": dict(B=2, dk=64, dv=128, dtype="f32", lens=[2, 18], cap=24),
    "kda": dict(B=3, gate="kda", lens=[0, 16, 33], cap=40),
    "kda shared": dict(B=4, gate="kda", share=2, H=4, Hqk=2, dk=64, dv=64, lens=[1, 2, 17, 0], cap=20),
    "kda strong": dict(B=2, gate="kda", lens=[17, 40], cap=40, dist="strong"),
    "kda wide": dict(B=1, H=1, dv=256, gate="kda", lens=[18], cap=20),
    "kda many heads": dict(B=32, H=32, gate="kda", lens=[i % 4 for i in range(31)] + [18], cap=18),
    "kda many wide heads": dict(B=16, H=64, Hqk=32, dv=256, gate="kda", lens=[i % 3 for i in range(16)], cap=2),
    "many heads": dict(B=32, H=32, lens=[i % 3 for i in range(32)], cap=2),
}


@pytest.mark.parametrize("name", FOLDS)
def test_fold_matches_definition(name):
    st, _, _ = build(dict(FOLDS[name], T=1), 9)
    rh, rw = draft_ref.fold(st)
    before = snapshot(st)
    h_out = torch.full((st.B,) + tuple(st.h.shape[1:]), SENT, device="cuda")
    c_out = None if st.conv_state is None else torch.zeros(
        (st.B,) + tuple(st.conv_state.shape[1:]), dtype=st.conv_state.dtype, device="cuda")
    len_out = torch.full((st.B,), -1, dtype=torch.int32, device="cuda")
    assert st.fold(h_out, c_out, len_out) == 0
    torch.cuda.synchronize()
    assert rel_err(h_out.cpu().numpy(), rh) <= TOL
    if c_out is not None:
        assert torch.equal(c_out.cpu(), torch.from_numpy(rw).to(c_out.dtype))
    assert len_out.tolist() == [0] * st.B
    for n, t in before.items():
        assert torch.equal(bits(getattr(st, n)), bits(t)), n
    if st.share == 1:                                 # in place: the same bits, lengths cleared
        assert st.fold() == 0
        torch.cuda.synchronize()
        assert torch.equal(st.h, h_out) and st.len.tolist() == [0] * st.B
        if c_out is not None:
            assert torch.equal(st.conv_state, c_out)


@pytest.mark.parametrize("in_place", [False, True])
def test_fold_of_the_long_tapes_only(in_place):
    spec = spec_of(H=2)
    st = make(spec, 5, 12, [0, 3, 4, 5, 12], seed=11)
    rh, _ = draft_ref.fold(st)
    h0, c0 = st.h.clone(), st.conv_state.clone()
    if in_place:
        assert st.fold(min_len=4) == 0
        got, lens = st.h, st.len
    else:
        got, lens = h0.clone(), torch.zeros(5, dtype=torch.int32, device="cuda")
        conv = c0.clone()
        assert st.fold(got, conv, lens, min_len=4) == 0
    torch.cuda.synchronize()
    assert lens.tolist() == [0, 3, 0, 0, 0]
    assert torch.equal(got[:2], h0[:2])
    assert rel_err(got[2:].cpu().numpy(), rh[2:]) <= TOL
    if in_place:
        assert torch.equal(st.conv_state[:2], c0[:2])


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_draft_and_fold_follow_decode(gate):
    """Tokens drafted in uneven steps with a fold on the way end at the state, windows and
    outputs of as many decode steps."""
    spec = dataclasses.replace(inputs.decode_config(4), H=4, Hqk=2, gate=gate, gate_dist="uniform",
                               out_gate=True, seed=21)
    inp = inputs.make(spec)
    n = 40
    dec = Decode(inp, "cuda")
    st = Drafts(spec, 4, 24, inp["h0"], inp["conv_state"], inp["conv_w"], norm_w=inp["norm_w"])
    x, g, beta, z = rows_of(spec, 4 * n, 22, z=True)
    x4, g4, b4, z4 = (t.view(4, n, -1) for t in (x, g, beta, z))
    want = torch.empty(4, n, spec.H, spec.dv, device="cuda")
    for t in range(n):
        dec.z = z4[:, t].contiguous()
        gt = g4[:, t].reshape(4, *g.shape[1:]).contiguous()
        assert dec.step(x4[:, t].contiguous(), 0, 1, gt, b4[:, t].contiguous()) == 0
        want[:, t] = dec.o
    t = 0
    for step, T in enumerate((1, 5, 16, 2, 1, 7, 8)):
        o = torch.empty(4 * T, spec.H, spec.dv, device="cuda")
        if int(st.len[0]) + T > st.cap:
            assert st.fold() == 0
        assert st.draft(x4[:, t:t + T].reshape(4 * T, -1).contiguous(),
                        g4[:, t:t + T].reshape(4 * T, *g.shape[1:]).contiguous(),
                        b4[:, t:t + T].reshape(4 * T, -1).contiguous(), o, T,
                        z=z4[:, t:t + T].reshape(4 * T, -1).contiguous()) == 0
        st.len += T
        ref = want[:, t:t + T].reshape(4 * T, spec.H, spec.dv)
        assert float((o - ref).abs().max()) <= 2 * TOL * 10 * float(ref.abs().max()), step
        t += T
    assert t == n and st.fold() == 0
    torch.cuda.synchronize()
    assert rel_err(st.h.cpu().numpy(), dec.h.cpu().numpy()) <= 2 * TOL
    assert torch.equal(st.conv_state, dec.conv_state)


def test_offsets_past_32_bits():
    """Tapes of more than 2^31 values: the last stream's entries lie past 32-bit offsets."""
    spec = spec_of(H=32)
    cap = 300000
    st = make(spec, 2, 4, [3, 2], seed=31, fill=0.0)
    small = {n: getattr(st, n) for n in ("k", "d", "g", "raw")}
    x, g, beta, _ = rows_of(spec, 4, 32)
    o, o2 = torch.empty(2, 4, 32, 128, device="cuda")
    h1, h2 = torch.empty(2, 2, 32, 128, 128, device="cuda")
    c1, c2 = torch.empty((2,) + tuple(st.conv_state.shape), dtype=torch.bfloat16, device="cuda")
    l1 = torch.empty(2, dtype=torch.int32, device="cuda")
    st.len.copy_(torch.tensor([2, 2], dtype=torch.int32))
    assert st.draft(x, g, beta, o, 2) == 0
    assert st.fold(h1, c1, l1) == 0
    for n, t in small.items():
        big = torch.zeros((2, cap) + tuple(t.shape[2:]), dtype=t.dtype, device="cuda")
        big[:, :2] = t[:, :2]
        setattr(st, n, big)
    st.cap = cap
    assert st.d.numel() > 2 ** 31
    assert st.draft(x, g, beta, o2, 2) == 0
    assert st.fold(h2, c2, l1) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(h1, h2) and torch.equal(c1, c2)
    for n, t in small.items():
        assert torch.equal(getattr(st, n)[:, :4], t), n


def test_two_calls_on_two_streams():
    """Calls on their own buffers need nothing of each other: two at once on two streams give
    what each gives alone."""
    spec = spec_of(H=4)
    runs, want = [], []
    for seed in (41, 42):
        st = make(spec, 8, 16, [i % 9 for i in range(8)], seed=seed, fill=0.0)
        rows = rows_of(spec, 8 * 4, seed + 10)
        o = torch.empty(32, 4, 128, device="cuda")
        assert st.draft(*rows[:3], o, 4) == 0
        torch.cuda.synchronize()
        want.append((o.clone(), st.d.clone()))
        o.zero_()
        runs.append((st, rows, o, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, rows, o, s in runs:
            assert st.draft(*rows[:3], o, 4, stream=s.cuda_stream) == 0
    torch.cuda.synchronize()
    for (st, _, o, _), (wo, wd) in zip(runs, want):
        assert torch.equal(o, wo) and torch.equal(st.d, wd)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_serving_loop_with_drafts(gate):
    """The three together, as a server runs them: the current token and its drafts go through
    gdn_draft, a head gives the target's probabilities, gdn_verify decides and moves the tapes
    on, gdn_fold empties the tapes that are nearly full. The tokens taken, run through a plain
    float64 pass, end at the same state."""
    spec = spec_of(H=2, gate=gate, dk=64, dv=64)
    B, T, V, cap, steps = 5, 4, 97, 14, 12
    st = make(spec, B, cap, [0] * B, seed=51, fill=float("nan"))
    h0, c0 = st.h.clone(), st.conv_state.clone()
    gen = torch.Generator(device="cuda").manual_seed(52)
    emb = torch.randn(V, spec.cd, generator=gen, device="cuda").to(torch.bfloat16)
    gshape = (2, 64) if gate == "kda" else (2,)
    gtab = -torch.rand(V, *gshape, generator=gen, device="cuda") * 0.3
    btab = torch.rand(V, 2, generator=gen, device="cuda")
    head = torch.randn(2 * 64, V, generator=gen, device="cuda")
    cur = torch.arange(B, device="cuda", dtype=torch.int32)
    taken = [[] for _ in range(B)]
    counts = []
    for step in range(steps):
        prop = torch.softmax(torch.randn(B, T, V, generator=gen, device="cuda"), -1)
        drafts = torch.multinomial(prop.view(B * T, V), 1, generator=gen).view(B, T).to(torch.int32)
        ids = torch.cat([cur[:, None], drafts], 1).long().view(-1)
        o = torch.empty(B * (T + 1), 2, 64, device="cuda")
        assert st.draft(emb[ids].contiguous(), gtab[ids].contiguous(), btab[ids].contiguous(), o, T + 1) == 0
        target = torch.softmax(o.view(B, T + 1, -1) @ head * 0.2, -1)
        u = torch.rand(B, T + 1, generator=gen, device="cuda")
        rc, acc, nxt = verify(target, drafts, u, draft=prop, len=st.len)
        assert rc == 0
        ra, rn = draft_ref.verify(target, drafts, u, draft=prop)
        assert acc.tolist() == ra.tolist() and nxt.tolist() == rn.tolist()
        for b in range(B):
            taken[b] += ids.view(B, T + 1)[b, :int(acc[b]) + 1].tolist()
        counts += acc.tolist()
        cur = nxt.clone()
        assert st.fold(min_len=cap - T) == 0
        assert int(st.len.max()) < cap - T
    assert st.fold() == 0
    torch.cuda.synchronize()
    assert 0 < sum(counts) < steps * B * T                      # some accepted, some refused
    for b in range(B):
        ids = torch.tensor(taken[b], device="cuda")
        one = Drafts(spec, 1, 1, h0[b:b + 1], c0[b:b + 1], st.conv_w)
        n = len(taken[b])
        _, rk, rd = draft_ref.draft(one, emb[ids], gtab[ids], btab[ids], n)
        ref = draft_ref.state_after(h0[b].double().cpu().numpy(), rk[0], rd[0],
                                    gtab[ids].double().cpu().numpy(), n, 1)
        assert rel_err(st.h[b].cpu().numpy(), ref) <= 2 * TOL
        assert torch.equal(st.conv_state[b].t(), torch.cat([c0[b].t(), emb[ids]])[-3:])


def test_step_in_a_graph():
    """draft, verify and fold captured once and replayed: every replay gives the eager result,
    with eager work and restored states between the replays."""
    spec = spec_of(H=2)
    B, T, V, cap = 6, 3, 501, 8
    st = make(spec, B, cap, [0, 1, 2, 3, 4, 5], seed=61, fill=0.0)
    x, g, beta, _ = rows_of(spec, B * (T + 1) - B, 62)
    gen = torch.Generator(device="cuda").manual_seed(63)
    target = torch.softmax(torch.randn(B, T + 1, V, generator=gen, device="cuda"), -1)
    prop = torch.softmax(torch.randn(B, T, V, generator=gen, device="cuda"), -1)
    toks = torch.randint(0, V, (B, T), generator=gen, device="cuda", dtype=torch.int32)
    u = torch.rand(B, T + 1, generator=gen, device="cuda")
    o = torch.empty(B * T, 2, 128, device="cuda")
    out = {}
    start = snapshot(st)

    def step():
        assert st.draft(x, g, beta, o, T) == 0
        rc, out["acc"], out["next"] = verify(target, toks, u, draft=prop, len=st.len)
        assert rc == 0
        assert st.fold(min_len=4) == 0

    def reset():
        for n, t in start.items():
            getattr(st, n).copy_(t)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    want = {**{n: t.clone() for n, t in snapshot(st).items()}, "o": o.clone(),
            "acc": out["acc"].clone(), "next": out["next"].clone()}
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        reset()
        o.fill_(float("nan"))
        torch.cuda.synchronize()
        torch.randn(1 << 20, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        got = {**snapshot(st), "o": o, **out}
        for n, t in want.items():
            assert torch.equal(bits(got[n]), bits(t)), (i, n)
