"""Plain attention with sinks, its gradient, and drafted trees in 64 bits, with bounds on what a kernel's roundings
may add (derived as in attend_util: the logits' error r |q|.|k| moves the weights, P is rounded by a relative p)."""
import numpy as np

from tests.attend_util import BF16


def attend_seen(q, k, v, seen, r, p):
    """q [n, d] scaled queries, k, v [m, d], seen [n, m], all in 64 bits -> output, bound, log-sum-exp.  A row that
    sees nothing is zero."""
    x = np.where(seen, q @ k.T, -np.inf)
    m = np.max(x, -1, keepdims=True, initial=-1e300)
    w = np.exp(x - m)
    total = w.sum(-1, keepdims=True)
    some = total > 0
    w /= np.where(some, total, 1)
    D = np.where(seen, r * (np.abs(q) @ np.abs(k).T), 0)
    o, size = w @ v, w @ np.abs(v)
    logits = (w * D) @ np.abs(v) + size * (w * D).sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(some, m + np.log(total), -np.inf)[:, 0]
    return o, BF16 * np.abs(o) + 1.1 * (logits + p * size) + 2.0 ** -12 * size, lse


def sink_seen(T, window, sinks):
    t, j = np.arange(T)[:, None], np.arange(T)[None]
    return (j <= t) & ((j > t - window) | (j < sinks))


def sink_fwd(x, k, v, alpha, beta, window, sinks, r=2.0 ** -11, p=BF16):
    """x [B, T, Hq, d] and k, v [B, T, Hkv, d] in 64 bits -> o, bound, lse."""
    B, T, Hq, d = x.shape
    G = Hq // k.shape[2]
    o, bound, lse = np.empty(x.shape), np.empty(x.shape), np.empty(x.shape[:3])
    seen = sink_seen(T, window, sinks)
    for b in range(B):
        for h in range(Hq):
            q = (x[b, :, h] * alpha[h] + beta[h]) * d ** -0.5
            o[b, :, h], bound[b, :, h], lse[b, :, h] = attend_seen(q, k[b, :, h // G], v[b, :, h // G], seen, r, p)
    return o, bound, lse


def sink_bwd(x, k, v, alpha, beta, dO, window, sinks, o=None, lse=None):
    """Gradients dx, dk, dv, dalpha, dbeta of sum(o * dO), by the chain rule; with o and lse (as the forward wrote
    them) the weights are exp(s - lse) and the rows' D is dO . o, as the library's gradient takes them."""
    B, T, Hq, d = x.shape
    G, scale = Hq // k.shape[2], d ** -0.5
    seen = sink_seen(T, window, sinks)
    dx, dk, dv = np.zeros(x.shape), np.zeros(k.shape), np.zeros(v.shape)
    da, db = np.zeros(alpha.shape), np.zeros(alpha.shape)
    for b in range(B):
        for h in range(Hq):
            kk, vv, g = k[b, :, h // G], v[b, :, h // G], dO[b, :, h]
            q = x[b, :, h] * alpha[h] + beta[h]
            s = np.where(seen, scale * (q @ kk.T), -np.inf)
            dp = g @ vv.T
            if lse is None:
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                D = (w * dp).sum(-1, keepdims=True)
            else:
                w, D = np.exp(s - lse[b, :, h, None]), (g * o[b, :, h]).sum(-1, keepdims=True)
            ds = w * (dp - D) * scale
            dq = ds @ kk
            dx[b, :, h] = dq * alpha[h]
            da[h] += (dq * x[b, :, h]).sum(0)
            db[h] += dq.sum(0)
            dk[b, :, h // G] += ds.T @ q
            dv[b, :, h // G] += w.T @ g
    return dx, dk, dv, da, db


def paths(parent):
    """The path of each node of one tree, root first; None below a bad parent."""
    out = []
    for i, up in enumerate(parent):
        if up == -1:
            out.append([i])
        elif 0 <= up < i and out[up] is not None:
            out.append(out[up] + [i])
        else:
            out.append(None)
    return out


def tree(x, xc, kn, vn, parent, k, v, lens, vec, window, sinks, nodes=None, r=2.0 ** -11, p=BF16):
    """x, xc [B, N, Hq, d], kn, vn [B, N, Hkv, d], k, v [B, L_max, Hkv, d] in 64 bits; vec: alpha, beta, alpha_c,
    beta_c -> (o, bound), (oc, bound); NaN in rows that are not written, zeros in those without a path."""
    B, N, Hq, d = x.shape
    G, scale = Hq // k.shape[2], d ** -0.5
    res = [[np.full(x.shape, np.nan) for _ in range(2)] for _ in range(2)]
    for b in range(B):
        n, L = N if nodes is None else nodes[b], lens[b]
        ways = paths(list(parent[b][:n]))
        pos = np.concatenate([np.arange(L), [L + len(w) - 1 if w else -1 for w in ways]]).astype(int)
        whole = np.zeros((n, L + n), bool)
        for i, w in enumerate(ways):
            if w:
                whole[i, :L] = True
                whole[i, L + np.array(w)] = True
        at = pos[L:, None]
        near = whole & ((pos[None] > at - window) | (pos[None] < sinks))
        for h in range(Hq):
            kk = np.concatenate([k[b, :L, h // G], kn[b, :n, h // G]])
            vv = np.concatenate([v[b, :L, h // G], vn[b, :n, h // G]])
            for s, (y, al, be, seen) in enumerate(((x, vec[0], vec[1], near), (xc, vec[2], vec[3], whole))):
                q = (y[b, :n, h] * al[h] + be[h]) * scale
                res[s][0][b, :n, h], res[s][1][b, :n, h], _ = attend_seen(q, kk, vv, seen, r, p)
    return res
