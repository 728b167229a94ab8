"""Timed cases of the serving operators that work on drafted tokens, each in a plain torch
form and, where ``own`` is set, through libgdn.

* draft  -- T new tokens per stream against states that are left as they are; what the
  tokens would add to the state goes onto the stream's tape. ``share`` consecutive streams
  read one state (a prefix computed once for all of them).
* fold   -- the entries of the tapes are worked into the states (and the carried windows).
* verify -- drafted tokens against the target's probabilities, from given random numbers,
  and the token that follows the accepted ones.

A stream's tape holds, per token it has taken since its state was written, the normalised
key k (per q/k head), the log-gate g, the update d (per value head) and the raw conv inputs.
With h the state in memory, the state after entry i is
    h_i = diag(e^(g_1+..+g_i)) h + sum_{j<=i} diag(e^(g_{j+1}+..+g_i)) k_j d_j^T.
"""
import math

import torch

own = False

WIN_STD, H0_STD = 1.0, 0.1


# ---- cases ------------------------------------------------------------------------------

def _draft(name, **kw):
    c = dict(op="draft", name=name, B=1, T=1, share=1, H=32, Hqk=32, dk=128, dv=128,
             dtype="bf16", gate="gdn", gates="uniform", conv_k=4, cap=16, nmin=0, nmax=12, z=False)
    c.update(kw)
    return c


def _fold(name, **kw):
    c = dict(op="fold", name=name, B=1, share=1, H=32, Hqk=32, dk=128, dv=128, dtype="bf16",
             gate="gdn", gates="uniform", conv_k=4, cap=16, nmin=1, nmax=16, min_len=1)
    c.update(kw)
    return c


def _verify(name, **kw):
    c = dict(op="verify", name=name, B=1, T=4, V=32000, dtype="f32", proposal=True,
             ragged=False, noise=0.5)
    c.update(kw)
    return c


def listed():
    return [
        # one user's stream, one token at a time: latency alone
        _draft("draft one token", H=32, Hqk=16, z=True),
        # a served batch, the current token and 4 drafted ones for each of 64 streams
        _draft("draft batch", B=64, T=5, cap=24, nmax=16),
        # the per-key-channel gate with the output gate, 3 drafted tokens
        _draft("draft channel gates", B=32, T=4, gate="kda", gates="slow", cap=24, nmax=20, z=True),
        # a small float32 model without the conv, odd counts
        _draft("draft float32", B=7, T=3, H=6, Hqk=2, dk=64, dv=64, dtype="f32", conv_k=0,
               cap=13, nmax=9),
        # 32 samples of each of 4 prompts: one prompt state per 32 streams
        _draft("draft shared prefix", B=128, T=2, share=32, H=32, Hqk=16, cap=32, nmax=16, gates="slow"),
        # the largest batch, 8 tokens per stream
        _draft("draft large", B=256, T=8, cap=32, nmax=16),
        # one stream's tape into its state
        _fold("fold one stream", Hqk=16),
        # a served batch, tapes of 1 to 16 tokens
        _fold("fold batch", B=64),
        # samples of a prompt leave the shared state for states of their own
        _fold("fold shared prefix", B=48, share=16, gate="kda", gates="slow", cap=40, nmax=33),
        # one stream, the smallest call
        _verify("verify one stream"),
        # drafts chosen without probabilities (looked up, or the likeliest token), odd vocabulary
        _verify("verify looked-up drafts", B=19, T=7, V=50257, proposal=False, ragged=True, dtype="bf16"),
        # a served batch, bf16 probabilities of a large vocabulary
        _verify("verify batch", B=256, T=4, V=131072, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["draft", "draft", "draft", "fold", "fold", "verify", "verify"])
    if op == "verify":
        V = _log(rng, 300, 200000)
        T = rng.randint(1, 8)
        B = _log(rng, 1, max(1, min(256, 256 * 4 * 131072 // (T * V))))
        return _undraw(_verify("", B=B, T=T, V=V, dtype=rng.choice(["f32", "bf16"]),
                               proposal=rng.random() < 0.75, ragged=rng.random() < 0.5,
                               noise=rng.choice([0.1, 0.5, 2.0])))
    dtype, dk, dv = rng.choice([("bf16", 128, 128)] * 3 + [("bf16", 64, 64), ("bf16", 128, 256),
                                                           ("f32", 64, 64), ("f32", 64, 128)])
    gate = rng.choice(["gdn", "gdn", "kda"])
    Hqk = _log(rng, 1, 32)
    H = Hqk * rng.choice([r for r in (1, 1, 2, 3, 4) if Hqk * r <= 48])
    top = 256 * 32 * 128 * 128 // (H * dk * dv * 2)      # at most half the largest batch
    share = rng.choice([1, 1, 1, rng.randint(2, 32)])
    kw = dict(share=share, H=H, Hqk=Hqk, dk=dk, dv=dv, dtype=dtype, gate=gate,
              gates=rng.choice(["uniform", "slow", "softplus"]), conv_k=rng.choice([0, 2, 3, 4, 4]))
    if op == "draft":
        T = rng.randint(1, 16) if rng.random() < 0.3 else rng.randint(1, 6)
        nmax = rng.choice([0, rng.randint(1, 16), rng.randint(1, 70)])
        cap = nmax + T + rng.randint(0, 9)
        if gate == "kda":                                 # the plain form's [T][cap+T][dk] products
            top = min(top, (1 << 28) // (H * T * (cap + T) * dk))
        groups = _log(rng, 1, max(1, min(256, top) // share))
        return _undraw(_draft("", B=groups * share, T=T, cap=cap, nmax=nmax, nmin=rng.randint(0, nmax),
                              z=rng.random() < 0.4, **kw))
    nmax = rng.randint(1, 16) if rng.random() < 0.5 else rng.randint(1, 70)
    groups = _log(rng, 1, max(1, min(256, top) // share))
    return _undraw(_fold("", B=groups * share, cap=nmax + rng.randint(0, 5), nmax=nmax,
                         nmin=rng.randint(0, nmax), min_len=rng.choice([0, 1, 1, max(1, nmax // 2)]), **kw))


def _undraw(c):
    del c["name"]
    return c


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _cd(c):
    return 2 * c["Hqk"] * c["dk"] + c["H"] * c["dv"]


def _lens(c):
    """Tape lengths from nmin to nmax, evenly spread over the streams."""
    B, lo, hi = c["B"], c["nmin"], c["nmax"]
    return [lo + (i * (hi - lo + 1)) // B if B > 1 else (lo + hi) // 2 for i in range(B)]


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "verify":
        # the target's row after the accepted drafts, once; the proposal's where one is refused
        # (about half of the streams)
        return {"bytes": c["B"] * c["V"] * es * (1.5 if c["proposal"] else 1.0),
                "flops": c["B"] * c["V"] * 3}
    B, H, Hqk, dk, dv, cd = c["B"], c["H"], c["Hqk"], c["dk"], c["dv"], _cd(c)
    K, gw = c["conv_k"], (c["dk"] if c["gate"] == "kda" else 1)
    state, entry, win = H * dk * dv * 4, 4 * (Hqk * dk + H * dv + H * gw), cd * max(K - 1, 0) * es
    lens = _lens(c)
    if c["op"] == "draft":
        T = c["T"]
        b = (B // c["share"]) * state + sum(lens) * entry               # states and tapes read
        b += B * T * (cd * es + 4 * H * (gw + 1) + 4 * H * dv)          # rows, gates, betas, o
        b += B * T * (entry + (cd * es if K else 0))                    # new entries
        b += (cd * K * 4 if K else 0) + sum(min(n, K - 1) * cd * es for n in lens if K)
        b += (B // c["share"]) * win if any(n < K - 1 for n in lens) else 0
        b += B * T * H * dv * es if c["z"] else 0
        f = sum(2 * T * 2 * H * (dk * dv + (n + (T + 1) / 2) * (dk + dv)) for n in lens)
        return {"bytes": b, "flops": f}
    on = [n for n in lens if n >= c["min_len"]]
    groups = len({i // c["share"] for i, n in enumerate(lens) if n >= c["min_len"]})
    b = groups * (state + win) + len(on) * (state + win) + sum(on) * entry
    b += sum(min(n, max(K - 1, 0)) * cd * es for n in on) + 8 * B
    return {"bytes": max(b, 1), "flops": sum(H * dk * dv * (2 * n + 1) for n in on)}


# ---- inputs -----------------------------------------------------------------------------

def _gates(c, gen, *shape):
    if c["gates"] == "softplus":
        x = torch.randn(*shape, generator=gen, device="cuda")
        return -torch.log1p(torch.exp(x))
    lo, hi = (-0.5, -0.01) if c["gates"] == "uniform" else (-0.02, -1e-4)
    return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    td = _dtype(c)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = {"case": c}
    B = c["B"]
    if c["op"] == "verify":
        T, V = c["T"], c["V"]
        logits = normal(B, T + 1, V, std=3.0)
        s["target"] = torch.softmax(logits, -1).to(td)
        drafted = torch.softmax(logits[:, :T] + c["noise"] * normal(B, T, V), -1).to(td)
        del logits
        if c["proposal"]:
            s["draft"] = drafted
            s["tokens"] = torch.stack([torch.multinomial(drafted[:, t].float(), 1, generator=gen)[:, 0]
                                       for t in range(T)], 1).to(torch.int32)
        else:
            s["draft"] = None
            s["tokens"] = drafted.argmax(-1).to(torch.int32)
        s["num"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda",
                                 dtype=torch.int32) if c["ragged"] else None
        s["u"] = torch.rand(B, T + 1, generator=gen, device="cuda")
        s["accepted"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["next"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s

    H, Hqk, dk, dv, K, cap, cd = c["H"], c["Hqk"], c["dk"], c["dv"], c["conv_k"], c["cap"], _cd(c)
    P = B // c["share"]
    gshape = (H, dk) if c["gate"] == "kda" else (H,)
    s["h"] = normal(P, H, dk, dv, std=H0_STD)
    s["h_ptrs"] = _ptrs(s["h"])
    s["conv"] = normal(P, cd, K - 1, std=WIN_STD, dtype=td) if K else None
    s["conv_ptrs"] = _ptrs(s["conv"]) if K else None
    s["conv_w"] = normal(cd, K, std=0.5) if K else None
    k = normal(B, cap, Hqk, dk)
    s["tape_k"] = k / k.square().sum(-1, keepdim=True).sqrt()
    s["tape_d"] = normal(B, cap, H, dv, std=0.5)
    s["tape_g"] = _gates(c, gen, B, cap, *gshape)
    s["tape_raw"] = normal(B, cap, cd, dtype=td) if K else None
    lens = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    s["len"] = lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()
    if c["op"] == "fold":
        s["h_out"] = torch.zeros(B, H, dk, dv, device="cuda")
        s["h_out_ptrs"] = _ptrs(s["h_out"])
        s["conv_out"] = torch.zeros(B, cd, K - 1, dtype=td, device="cuda") if K else None
        s["conv_out_ptrs"] = _ptrs(s["conv_out"]) if K else None
        s["len_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    T = c["T"]
    s["x"] = normal(B * T, cd, dtype=td)
    s["g"] = _gates(c, gen, B * T, *gshape)
    s["beta"] = torch.sigmoid(normal(B * T, H))
    s["o"] = torch.zeros(B * T, H, dv, device="cuda")
    s["z"] = normal(B * T, H, dv, dtype=td) if c["z"] else None
    s["norm_w"] = torch.rand(dv, generator=gen, device="cuda") + 0.5 if c["z"] else None
    return s


def _ptrs(t):
    return torch.tensor([t[i].data_ptr() for i in range(t.shape[0])], dtype=torch.int64, device="cuda")


# ---- the framework's calls --------------------------------------------------------------

def _own_params(s):
    """The parameter blocks of the calls on this state's buffers, as a serving loop keeps them."""
    from gated_delta_rule_depthwise_amd import binding as G
    c = s["case"]
    p = G.params(c["H"], c["dk"], c["dv"], dtype=G.GDN_BF16 if c["dtype"] == "bf16" else G.GDN_F32,
                 conv_k=c["conv_k"], ld_qkv=_cd(c), Hqk=c["Hqk"], z=s.get("z"), norm_w=s.get("norm_w"))
    return p, G.tape(s["tape_k"], s["tape_d"], s["tape_g"], s["tape_raw"], s["len"], c["cap"])


def _own(s):
    from gated_delta_rule_depthwise_amd import binding as G
    c = s["case"]
    stream = torch.cuda.current_stream().cuda_stream
    if c["op"] == "verify":
        if "ws" not in s:
            n = G.gdn_verify_workspace_bytes(c["B"], c["T"], c["V"])
            s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
            s["ws_bytes"] = n
        rc = G.gdn_verify(s["target"], c["V"], s["draft"], c["V"],
                          G.GDN_BF16 if c["dtype"] == "bf16" else G.GDN_F32, s["tokens"], s["num"], s["u"],
                          c["B"], c["T"], c["V"], s["accepted"], s["next"], None, s["ws"], s["ws_bytes"], stream)
        out = {"accepted": s["accepted"], "next": s["next"]}
    else:
        if "blocks" not in s:
            s["blocks"] = _own_params(s)
        p, tape = s["blocks"]
        kda = c["gate"] == "kda"
        if c["op"] == "draft":
            x, es = s["x"].data_ptr(), s["x"].element_size()
            fn = G.kda_draft if kda else G.gdn_draft
            rc = fn(p, x, x + c["Hqk"] * c["dk"] * es, x + 2 * c["Hqk"] * c["dk"] * es, s["g"], s["beta"],
                    s["h_ptrs"], s["conv_ptrs"], s["conv_w"], tape, s["o"], c["B"], c["T"], c["share"], stream)
            out = _draft_out(s)
        else:
            fn = G.kda_fold if kda else G.gdn_fold
            rc = fn(p, s["h_ptrs"], s["conv_ptrs"], s["h_out_ptrs"], s["conv_out_ptrs"], tape, s["len_out"],
                    c["B"], c["share"], c["min_len"], stream)
            out = _fold_out(s)
    if rc != 0:
        raise RuntimeError("libgdn: " + G.gdn_status_string(rc))
    return out


def _draft_out(s):
    out = {"o": s["o"], "k": s["tape_k"], "d": s["tape_d"], "g": s["tape_g"]}
    if s["tape_raw"] is not None:
        out["raw"] = s["tape_raw"]
    return out


def _fold_out(s):
    out = {"h": s["h_out"], "len": s["len_out"]}
    if s["conv_out"] is not None:
        out["conv"] = s["conv_out"]
    return out


# ---- plain forms ------------------------------------------------------------------------

def _windows(s, dtype):
    """[B][K-1][cd]: the raw inputs before each stream's next token, oldest first: from the
    tape, and from the carried window where the tape is shorter."""
    c = s["case"]
    W, B = c["conv_k"] - 1, c["B"]
    m = s["len"].long()[:, None] - W + torch.arange(W, device="cuda")[None, :]
    tape = s["tape_raw"][torch.arange(B, device="cuda")[:, None], m.clamp(min=0)].to(dtype)
    win = s["conv"].to(dtype).transpose(1, 2).repeat_interleave(c["share"], 0)       # [B][W][cd]
    win = win.gather(1, (W + m).clamp(max=W - 1)[:, :, None].expand(B, W, win.shape[2]))
    return torch.where((m >= 0)[:, :, None], tape, win)


def _heads(x, c):
    """q/k heads repeated for the value heads they serve, at the heads' axis -2."""
    return x.repeat_interleave(c["H"] // c["Hqk"], -2)


def _plain_draft(s):
    c = s["case"]
    B, T, H, Hqk, dk, dv, cap, K = (c[n] for n in ("B", "T", "H", "Hqk", "dk", "dv", "cap", "conv_k"))
    n = s["len"].long()
    x = s["x"].view(B, T, -1).float()
    if K:
        seq = torch.cat([_windows(s, torch.float32), x], 1)
        y = (seq.unfold(1, K, 1) * s["conv_w"]).sum(-1)
        x = y / (1 + torch.exp(-y))
    q, k, v = x.split([Hqk * dk, Hqk * dk, H * dv], -1)
    q, k, v = q.reshape(B, T, Hqk, dk), k.reshape(B, T, Hqk, dk), v.reshape(B, T, H, dv)
    q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6) * dk ** -0.5
    k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
    g = s["g"].view(B, T, *s["g"].shape[1:])
    beta = s["beta"].view(B, T, H)
    # log-decays from the state in memory through each tape entry in use and each new token
    used = torch.arange(cap, device="cuda")[None] < n[:, None]                        # [B][cap]
    tg = torch.where(used.view(B, cap, *([1] * (g.dim() - 2))), s["tape_g"], 0.0)
    cum = torch.cat([tg, g], 1).double().cumsum(1)
    cum = cum.transpose(1, 2)                                                        # [B][H][cap+T](dk)
    kq = torch.cat([_heads(k, c), _heads(q, c)], 1).transpose(1, 2)                  # [B][H][2T][dk]
    keys = torch.cat([_heads(s["tape_k"], c), _heads(k, c)], 1).transpose(1, 2)      # [B][H][cap+T][dk]
    now, two = cum[:, :, cap:], torch.cat([cum[:, :, cap:]] * 2, 2)                  # the new tokens, for k and q
    h = s["h"]
    P = h.shape[0]
    t = torch.arange(T, device="cuda")
    j = torch.arange(cap + T, device="cuda") - cap
    seen = torch.where((j < 0)[None, None, :], used.repeat(1, 2 * T).view(B, 2 * T, cap)[:, :, (j + cap).clamp(max=cap - 1)],
                       (j[None, :] < torch.cat([t, t + 1])[:, None])[None])          # k_t: j < t, q_t: j <= t
    if g.dim() == 4:
        decay = torch.exp((two[:, :, :, None] - cum[:, :, None]).float())
        a = (kq[:, :, :, None] * keys[:, :, None] * torch.where(seen[:, None, :, :, None], decay, 0.0)).sum(-1)
        base = kq * torch.exp(two.float())
    else:
        decay = torch.exp(torch.where(seen[:, None], two[..., None] - cum[:, :, None], 0.0).float())
        a = torch.where(seen[:, None], (kq @ keys.transpose(-1, -2)) * decay, 0.0)
        base = kq * torch.exp(two.float())[..., None]
    # the streams of one state side by side, so that the state is read once for all of them
    base = base.view(P, -1, H, 2 * T, dk).transpose(1, 2).reshape(P, H, -1, dk) @ h
    base = base.view(P, H, -1, 2 * T, dv).transpose(1, 2).reshape(B, H, 2 * T, dv)
    td = torch.where(used[:, :, None, None], s["tape_d"], 0.0).transpose(1, 2)       # [B][H][cap][dv]
    base = base + a[..., :cap] @ td
    bt = beta.transpose(1, 2)[..., None]
    rhs = (bt * (v.transpose(1, 2) - base[:, :, :T])).double()
    # d = (I + N)^-1 rhs, N strictly lower triangular: (I - N)(I + N^2)(I + N^4)(I + N^8)
    N = (bt * a[:, :, :T, cap:]).double()
    N2 = N @ N
    N4 = N2 @ N2
    d = rhs - N @ rhs
    d = d + N2 @ d
    d = d + N4 @ d
    d = (d + N4 @ (N4 @ d)).float()
    o = base[:, :, T:] + a[:, :, T:, cap:] @ d
    o, d = o.transpose(1, 2), d.transpose(1, 2)                                      # [B][T][H][dv]
    if s["z"] is not None:
        z = s["z"].view(B, T, H, dv).float()
        o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + 1e-6) * s["norm_w"] * z / (1 + torch.exp(-z))
    s["o"].copy_(o.reshape(B * T, H, dv))
    at = (torch.arange(B, device="cuda")[:, None], n[:, None] + t[None])
    s["tape_k"][at] = k
    s["tape_d"][at] = d
    s["tape_g"][at] = g
    if K:
        s["tape_raw"][at] = s["x"].view(B, T, -1)
    return _draft_out(s)


def _plain_fold(s):
    c = s["case"]
    B, H, cap, share = c["B"], c["H"], c["cap"], c["share"]
    n = s["len"].long()
    on = n >= c["min_len"]
    used = torch.arange(cap, device="cuda")[None] < n[:, None]
    tg = torch.where(used.view(B, cap, *([1] * (s["tape_g"].dim() - 2))), s["tape_g"], 0.0)
    cum = tg.double().cumsum(1)
    total = cum[:, -1:]
    left = torch.exp((total - cum).float())                                          # decay after each entry
    through = torch.exp(total.float())
    k = _heads(s["tape_k"], c)
    k = torch.where(used[:, :, None, None], k * (left if left.dim() == 4 else left[..., None]), 0.0)
    d = torch.where(used[:, :, None, None], s["tape_d"], 0.0)
    h = s["h"].repeat_interleave(share, 0) * through[:, 0].reshape(B, H, -1, 1)
    h = h + k.permute(0, 2, 3, 1) @ d.transpose(1, 2)
    s["h_out"].copy_(torch.where(on[:, None, None, None], h, s["h_out"]))
    if c["conv_k"]:
        win = _windows(s, s["conv"].dtype).transpose(1, 2)
        s["conv_out"].copy_(torch.where(on[:, None, None], win, s["conv_out"]))
    s["len_out"].copy_(torch.where(on, 0, n))
    return _fold_out(s)


def _plain_verify(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    b = torch.arange(B, device="cuda")
    num = s["num"].long() if s["num"] is not None else torch.full((B,), T, device="cuda")
    tok = s["tokens"].long()
    p = s["target"][:, :T].gather(2, tok[..., None])[..., 0].double()
    q = s["draft"].gather(2, tok[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p)
    ok = (s["u"][:, :T].double() * q < p) & (torch.arange(T, device="cuda")[None] < num[:, None])
    a = ok.int().cumprod(1).sum(1)
    row = s["target"][b, a].float()
    at = a.clamp(max=T - 1)
    if s["draft"] is not None:
        rest = (row - s["draft"][b, at].float()).clamp(min=0)
    else:
        one = torch.arange(V, device="cuda")[None] == tok[b, at][:, None]
        rest = torch.where(one, (row - 1).clamp(min=0), row)
    rest = torch.where((a < num)[:, None], rest, row)
    cum = rest.double().cumsum(1)
    cum = torch.where(cum[:, -1:] > 0, cum, row.double().cumsum(1))
    aim = s["u"][b, T].double() * cum[:, -1]
    s["next"].copy_((cum <= aim[:, None]).sum(1))
    s["accepted"].copy_(a)
    return {"accepted": s["accepted"], "next": s["next"]}


def run(state):
    if own:
        return _own(state)
    return {"draft": _plain_draft, "fold": _plain_fold, "verify": _plain_verify}[state["case"]["op"]](state)


# ---- the definition, token by token in 64 bits --------------------------------------------

def exact(case, seed):
    c = dict(case)
    if c["op"] == "verify":
        return None                                       # whole numbers only
    s = prepare(c, seed)
    B, H, Hqk, dk, dv, cap, K = (c[n] for n in ("B", "H", "Hqk", "dk", "dv", "cap", "conv_k"))
    n = s["len"].tolist()
    rep, W = H // Hqk, max(K - 1, 0)
    h = s["h"].double().repeat_interleave(c["share"], 0)

    def column(g):                                        # e^g as a factor of h's rows
        return torch.exp(g.double()).reshape(B, H, -1, 1)

    def outer(k, d):
        return k.repeat_interleave(rep, 1)[..., None] * d[:, :, None]

    for i in range(max(n)):
        live = (s["len"] > i)[:, None, None, None]
        h = torch.where(live, h * column(s["tape_g"][:, i])
                        + outer(s["tape_k"][:, i].double(), s["tape_d"][:, i].double()), h)
    if K:
        past = []
        for b in range(B):
            both = torch.cat([s["conv"][b // c["share"]].t(), s["tape_raw"][b, :n[b]]])
            past.append(both[both.shape[0] - W:])
        past = torch.stack(past)                          # [B][W][cd]
    if c["op"] == "fold":
        on = s["len"] >= c["min_len"]
        out = {"h": torch.where(on[:, None, None, None], h, 0.0), "len": None}
        if K:
            out["conv"] = torch.where(on[:, None, None], past.double().transpose(1, 2), 0.0)
        return out
    T = c["T"]
    x = s["x"].view(B, T, -1).double()
    if K:
        x = torch.cat([past.double(), x], 1)
    w = s["conv_w"].double() if K else None
    tapes = {"k": s["tape_k"].double(), "d": s["tape_d"].double(), "g": s["tape_g"].double()}
    outs = []
    for t in range(T):
        if K:
            y = torch.zeros_like(x[:, 0])
            for i in range(K):
                y = y + w[:, i] * x[:, t + i]
            y = y * torch.sigmoid(y)
        else:
            y = x[:, t]
        q, k = y[:, :Hqk * dk].view(B, Hqk, dk), y[:, Hqk * dk:2 * Hqk * dk].view(B, Hqk, dk)
        v = y[:, 2 * Hqk * dk:].view(B, H, dv)
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6) / math.sqrt(dk)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
        g = s["g"].view(B, T, *s["g"].shape[1:])[:, t]
        beta = s["beta"].view(B, T, H)[:, t].double()
        h = h * column(g)
        told = (k.repeat_interleave(rep, 1)[..., None] * h).sum(2)
        d = beta[..., None] * (v - told)
        h = h + outer(k, d)
        o = (q.repeat_interleave(rep, 1)[..., None] * h).sum(2)
        if c["z"]:
            z = s["z"].view(B, T, H, dv)[:, t].double()
            o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * s["norm_w"].double() * z * torch.sigmoid(z)
        outs.append(o)
        for b in range(B):
            tapes["k"][b, n[b] + t] = k[b]
            tapes["d"][b, n[b] + t] = d[b]
            tapes["g"][b, n[b] + t] = g[b].double()
    out = {"o": torch.stack(outs, 1).reshape(B * T, H, dv), **tapes}
    if K:
        raw = s["tape_raw"].double()
        for b in range(B):
            raw[b, n[b]:n[b] + T] = s["x"].view(B, T, -1)[b].double()
        out["raw"] = raw
    return out
