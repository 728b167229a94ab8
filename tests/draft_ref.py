"""The steps on drafted tokens in float64, token by token from their definition (numpy, one
stream and head at a time): the reference of the GPU tests. Shares no code with the library."""
import numpy as np


def _f64(x):
    return None if x is None else x.detach().cpu().double().numpy()


def state_after(h, k, d, g, n, rep):
    """h [H, dk, dv] after n tape entries: k [cap, Hqk, dk], d [cap, H, dv], g [cap, H(, dk)]."""
    h = h.copy()
    for i in range(n):
        for hd in range(h.shape[0]):
            h[hd] *= np.exp(g[i, hd]).reshape(-1, 1)
            h[hd] += np.outer(k[i, hd // rep], d[i, hd])
    return h


def window_after(win, raw, n):
    """[cd, K-1] raw inputs after n tape entries."""
    if win is None:
        return None
    both = np.concatenate([win.T, raw[:n]], 0)
    return both[both.shape[0] - win.shape[1]:].T


def draft(st, x, g, beta, T, z=None):
    """``st`` is a runner.Drafts (its tapes before the call); returns o [B*T, H, dv] and, per
    stream, the new entries k [T, Hqk, dk], d [T, H, dv]."""
    sp = st.spec
    H, Hqk, dk, dv = sp.H, sp.qk_heads, sp.dk, sp.dv
    rep = H // Hqk
    hs, cs, cw = _f64(st.h), _f64(st.conv_state), _f64(st.conv_w)
    tk, td, tg, tr = (_f64(t) for t in (st.k, st.d, st.g, st.raw))
    x, g, beta, z, nw = (_f64(t) for t in (x, g, beta, z, st.norm_w))
    lens = st.len.cpu().tolist()
    o = np.zeros((st.B * T, H, dv))
    ks, ds = np.zeros((st.B, T, Hqk, dk)), np.zeros((st.B, T, H, dv))
    for b in range(st.B):
        n, p = lens[b], b // st.share
        h = state_after(hs[p], tk[b], td[b], tg[b], n, rep)
        rows = x[b * T:(b + 1) * T, :sp.cd]
        if cw is not None:
            K = cw.shape[1]
            seq = np.concatenate([window_after(cs[p], tr[b], n).T, rows], 0)
            y = sum(cw[:, i] * seq[i:i + T] for i in range(K))
            rows = y / (1 + np.exp(-y))
        for t in range(T):
            q, k = rows[t, :Hqk * dk].reshape(Hqk, dk), rows[t, Hqk * dk:2 * Hqk * dk].reshape(Hqk, dk)
            v = rows[t, 2 * Hqk * dk:].reshape(H, dv)
            if st.eps >= 0:
                q = q / np.sqrt((q * q).sum(-1, keepdims=True) + st.eps)
                k = k / np.sqrt((k * k).sum(-1, keepdims=True) + st.eps)
            q = q * st.scale
            ks[b, t] = k
            for hd in range(H):
                r = b * T + t
                h[hd] *= np.exp(g[r, hd]).reshape(-1, 1)
                d = beta[r, hd] * (v[hd] - h[hd].T @ k[hd // rep])
                h[hd] += np.outer(k[hd // rep], d)
                ds[b, t, hd] = d
                out = h[hd].T @ q[hd // rep]
                if z is not None:
                    zz = z[r].reshape(H, dv)[hd]
                    out = out / np.sqrt(np.mean(out * out) + sp.norm_eps) * nw * zz / (1 + np.exp(-zz))
                o[r, hd] = out
    return o, ks, ds


def fold(st):
    """(h [B, H, dk, dv], windows [B, cd, K-1] or None) after every stream's tape."""
    sp = st.spec
    hs, cs = _f64(st.h), _f64(st.conv_state)
    tk, td, tg, tr = (_f64(t) for t in (st.k, st.d, st.g, st.raw))
    lens = st.len.cpu().tolist()
    h = np.stack([state_after(hs[b // st.share], tk[b], td[b], tg[b], lens[b], sp.H // sp.qk_heads)
                  for b in range(st.B)])
    w = None if cs is None else np.stack([window_after(cs[b // st.share], tr[b], lens[b])
                                          for b in range(st.B)])
    return h, w


def verify(target, tokens, u, draft=None, num=None):
    """(accepted [B], next [B]) from float64 sums taken in order."""
    p, q, u = _f64(target), _f64(draft), _f64(u)
    tokens = tokens.cpu().numpy()
    B, T1, V = p.shape
    T = T1 - 1
    acc, nxt = [], []
    for b in range(B):
        n = T if num is None else min(max(int(num[b]), 0), T)
        a = 0
        while a < n:
            t = int(tokens[b, a])
            if not 0 <= t < V:
                break
            qq = q[b, a, t] if q is not None else 1.0
            if not u[b, a] * qq < p[b, a, t]:
                break
            a += 1
        row = np.maximum(np.nan_to_num(p[b, a], nan=0.0), 0.0)
        r = row
        if a < n:
            t = int(tokens[b, a])
            if q is not None:
                other = q[b, a]
            else:
                other = np.zeros(V)
                if 0 <= t < V:
                    other[t] = 1.0
            # the difference is one rounding to float32 of the stored values
            d = (p[b, a].astype(np.float32) - other.astype(np.float32)).astype(np.float64)
            r = np.maximum(np.nan_to_num(d, nan=0.0), 0.0)
        cum = np.cumsum(r)
        if not cum[-1] > 0:
            r = row
            cum = np.cumsum(r)
        acc.append(a)
        if not cum[-1] > 0:
            nxt.append(-1)
            continue
        over = np.nonzero(cum > u[b, T] * cum[-1])[0]
        nxt.append(int(over[0]) if over.size else int(np.nonzero(r > 0)[0][-1]))
    return np.array(acc), np.array(nxt)
