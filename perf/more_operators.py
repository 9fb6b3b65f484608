"""Attention sinks and drafted trees: the cases that are measured, their plain forms, and the calls a
user makes.

* ``sink_fwd``: the base stream with a sliding window and a few first tokens that stay visible
  (sinks): row t attends over keys j <= t with j > t - window or j < sinks;
* ``sink_bwd``: its gradient, given the forward's output and log-sum-exp;
* ``tree``: both streams of a tree of drafted tokens over a cache.  Node i hangs below node
  parent[i] (-1: below the last cached token) and stands at position cache_len + depth; its copy
  attends over the cached rows and its ancestors with itself, its base token over those of them that
  lie in its window or among the sinks;
* ``accept``: the rows of the path that ends at an accepted node, appended to the cache.
"""
import math

import torch

own = False

_HEADS = ((2, 1, 64), (8, 2, 64), (4, 4, 64), (16, 1, 128), (8, 4, 128), (32, 8, 128))


def listed():
    q = {"Hq": 32, "Hkv": 8, "d": 128}
    s = {"Hq": 8, "Hkv": 2, "d": 64}
    return [
        # a 128K prompt of two sequences through the 8B-class layer
        {"name": "sink prefill 2x131072", "op": "sink_fwd", "B": 2, "T": 131072, "window": 128, "sinks": 4,
         "lse": False, **q},
        # the forward of a training step over four 16K sequences
        {"name": "sink training forward 4x16384", "op": "sink_fwd", "B": 4, "T": 16384, "window": 128, "sinks": 4,
         "lse": True, **q},
        # a short prompt on a small layer: latency counts
        {"name": "sink prefill 1x513", "op": "sink_fwd", "B": 1, "T": 513, "window": 128, "sinks": 4, "lse": False,
         "Hq": 2, "Hkv": 1, "d": 64},
        # a wide window with many sinks
        {"name": "sink prefill wide 1x8192", "op": "sink_fwd", "B": 1, "T": 8192, "window": 1024, "sinks": 16,
         "lse": False, **s},
        # the gradient of that training step
        {"name": "sink gradient 4x16384", "op": "sink_bwd", "B": 4, "T": 16384, "window": 128, "sinks": 4, **q},
        # the gradient of a small odd batch
        {"name": "sink gradient 3x500", "op": "sink_bwd", "B": 3, "T": 500, "window": 77, "sinks": 5, **s},
        # sixteen drafted tokens checked behind 128K prompts
        {"name": "tree 16 over 2x131072", "op": "tree", "B": 2, "L": 131072, "N": 16, "shape": "random",
         "window": 128, "sinks": 0, "ragged": False, **q},
        # wide trees for a batch of sequences of every length up to 16K
        {"name": "tree 64 over ragged 8x16384", "op": "tree", "B": 8, "L": 16384, "N": 64, "shape": "random",
         "window": 128, "sinks": 4, "ragged": True, **q},
        # a chain of five drafted tokens behind a short prompt: latency counts
        {"name": "tree 5 over 1x300", "op": "tree", "B": 1, "L": 300, "N": 5, "shape": "chain", "window": 128,
         "sinks": 0, "ragged": False, **s},
        # no draft: the single token of a decode step of a layer with sinks
        {"name": "tree 1 over 2x131072 sinks", "op": "tree", "B": 2, "L": 131072, "N": 1, "shape": "chain",
         "window": 128, "sinks": 4, "ragged": False, **q},
        # what the check of those wide trees accepted
        {"name": "accept 8 of 64", "op": "accept", "B": 8, "L": 16384, "N": 64, "shape": "random", **q},
        # accepted chains of a large batch
        {"name": "accept 64 of 8", "op": "accept", "B": 64, "L": 4096, "N": 8, "shape": "chain", **q},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sink_fwd", "sink_fwd", "sink_bwd", "tree", "tree", "accept"])
    Hq, Hkv, d = rng.choice(_HEADS)
    heads = {"Hq": Hq, "Hkv": Hkv, "d": d}
    window = rng.choice([1, 33, 77, 128, 128, 128, 300, 1000])
    if op in ("sink_fwd", "sink_bwd"):
        # values of q times window, and values of q, that a case may hold
        budget = min((1 << 28) * 128 // max(window, 128), 1 << 28 if op == "sink_bwd" else 1 << 30)
        B = _log(rng, 1, 8)
        T = _log(rng, 1, max(1, min(131072, budget // (B * Hq * d))))
        c = {"op": op, "B": B, "T": T, "window": window, "sinks": rng.choice([1, 2, 4, 4, 4, 8, 16, 27, 32]), **heads}
        if op == "sink_fwd":
            c["lse"] = rng.random() < 0.4
        return c
    N = _log(rng, 1, 64)
    shape = rng.choice(["chain", "random", "random", "wide"])
    if op == "accept":
        return {"op": op, "B": _log(rng, 1, 64), "L": _log(rng, 64, 8192), "N": N, "shape": shape, **heads}
    budget = 1 << 28  # values of K (and of V) in the cache, and logits
    B = _log(rng, 1, 32)
    L = _log(rng, 1, max(1, min(131072, budget // (B * Hkv * d), (1 << 29) // (B * Hq * N))))
    return {"op": op, "B": B, "L": L, "N": N, "shape": shape, "window": window, "sinks": rng.choice([0, 0, 1, 4, 16, 32]),
            "ragged": rng.random() < 0.6, **heads}


# ---------------------------------------------------------------------------------- inputs


def _normal(gen, *shape, dtype=torch.bfloat16):
    out = torch.empty(shape, device="cuda", dtype=dtype)
    for row in out.view((-1,) + shape[-3:]) if len(shape) > 3 else (out,):  # by sequences: a batch in 32 bits is large
        row.copy_(torch.randn(row.shape, generator=gen, device="cuda", dtype=torch.float32))
    return out


def _vectors(gen, Hq, d):
    one = torch.ones((Hq, d), device="cuda")
    return (one + 0.1 * _normal(gen, Hq, d, dtype=torch.float32), 0.1 * _normal(gen, Hq, d, dtype=torch.float32))


def _trees(gen, B, N, shape):
    """parent [B, N] int32: node i hangs below an earlier node, or below the cache (-1)."""
    i = torch.arange(N, device="cuda", dtype=torch.int32)[None].expand(B, N)
    if shape == "chain":
        return (i - 1).contiguous()
    u = torch.rand((B, N), generator=gen, device="cuda")
    if shape == "wide":  # most nodes below a few first ones
        return torch.minimum((u * u * (i + 1)).to(torch.int32) - 1, i - 1)
    return torch.minimum((u.sqrt() * (i + 1)).to(torch.int32) - 1, i - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, op = case, case["op"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    s = {"case": dict(c)}
    if op in ("sink_fwd", "sink_bwd"):
        T = c["T"]
        s["alpha"], s["beta"] = _vectors(gen, Hq, d)
        s["q"] = _normal(gen, B, T, Hq, d)
        s["k"], s["v"] = _normal(gen, B, T, Hkv, d), _normal(gen, B, T, Hkv, d)
        if op == "sink_bwd":
            s["dO"] = _normal(gen, B, T, Hq, d)
            s["o"], s["lse"] = _plain_sink_fwd(s, True)
        return s
    N, L_max = c["N"], (c["L"] + c["N"] + 127) // 128 * 128
    s["parent"] = _trees(gen, B, N, c["shape"])
    s["k_new"], s["v_new"] = _normal(gen, B, N, Hkv, d), _normal(gen, B, N, Hkv, d)
    s["k_cache"], s["v_cache"] = _normal(gen, B, L_max, Hkv, d), _normal(gen, B, L_max, Hkv, d)
    if op == "accept":
        s["lens"] = torch.randint(0, c["L"] + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["cache_len"] = s["lens"].clone()
        s["node"] = torch.randint(-1, N, (B,), generator=gen, device="cuda", dtype=torch.int32)
        return s
    s["alpha"], s["beta"] = _vectors(gen, Hq, d)
    s["alpha_c"], s["beta_c"] = _vectors(gen, Hq, d)
    s["q"], s["qc"] = _normal(gen, B, N, Hq, d), _normal(gen, B, N, Hq, d)
    s["cache_len"] = torch.full((B,), c["L"], device="cuda", dtype=torch.int32)
    s["nodes"] = None
    if c["ragged"]:  # the first sequence is the longest and has a full tree
        s["cache_len"] = torch.randint(0, c["L"] + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["nodes"] = torch.randint(0, N + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["cache_len"][0], s["nodes"][0] = c["L"], N
    s["o"], s["oc"] = _normal(gen, B, N, Hq, d), _normal(gen, B, N, Hq, d)  # rows behind a tree stay as they are
    return s


# ---------------------------------------------------------------------------------- plain forms

_ROWS = 128  # query rows of a block


def _some(n, cost):
    """Ranges of 0 .. n - 1 whose cost stays bounded."""
    step = max(1, int((1 << 30) // max(cost, 1)))
    return [(i, min(i + step, n)) for i in range(0, n, step)]


def _sink_parts(s, b):
    """For runs of blocks of sequence b: rows [n, _ROWS], queries [n, _ROWS, Hkv, G, d], keys of the
    window and their rows, logits [n, _ROWS, Hkv, G, window + _ROWS - 1] and of the sinks, masked."""
    c = s["case"]
    T, Hkv, d = c["T"], c["Hkv"], c["d"]
    w, ns = min(c["window"], T), min(c["sinks"], T)
    k, v = s["k"][b].float(), s["v"][b].float()
    total = (T + _ROWS - 1) // _ROWS
    for i0, i1 in _some(total, _ROWS * (w + _ROWS + ns) * c["Hq"]):
        j = torch.arange(i0, i1, device="cuda")[:, None] * _ROWS - w + 1 + torch.arange(w + _ROWS - 1, device="cuda")
        kb, vb = k[j.clamp(0, T - 1)], v[j.clamp(0, T - 1)]
        t = torch.arange(i0, i1, device="cuda")[:, None] * _ROWS + torch.arange(_ROWS, device="cuda")
        q = (s["q"][b][t.clamp(max=T - 1)].float() * s["alpha"] + s["beta"]).reshape(i1 - i0, _ROWS, Hkv, -1, d)
        scale = 1.0 / math.sqrt(d)
        x = torch.einsum("nrhgd,nkhd->nrhgk", q, kb) * scale
        y = torch.einsum("nrhgd,khd->nrhgk", q, k[:ns]) * scale
        tt, jj = t[:, :, None], j[:, None, :]
        seen = (jj <= tt) & (jj > tt - w) & (jj >= 0) & (tt < T)
        first = (torch.arange(ns, device="cuda") <= tt - w) & (tt < T)
        x.masked_fill_(~seen[:, :, None, None], -math.inf)
        y.masked_fill_(~first[:, :, None, None], -math.inf)
        yield t, q, kb, vb, j, x, y, k[:ns], v[:ns]


def _plain_sink_fwd(s, want_lse):
    c = s["case"]
    B, T, Hq, d = c["B"], c["T"], c["Hq"], c["d"]
    o = torch.empty((B, T, Hq, d), device="cuda", dtype=torch.bfloat16)
    lse = torch.empty((B, T, Hq), device="cuda") if want_lse else None
    for b in range(B):
        for t, q, kb, vb, j, x, y, ks, vs in _sink_parts(s, b):
            m = torch.maximum(x.amax(-1), y.amax(-1)).clamp(min=-1e30)[..., None]
            x, y = x.sub_(m).exp_(), y.sub_(m).exp_()
            total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
            out = torch.einsum("nrhgk,nkhd->nrhgd", x, vb) + torch.einsum("nrhgk,khd->nrhgd", y, vs)
            rows = (t < T).reshape(-1)
            flat = t.reshape(-1)[rows]
            o[b].index_copy_(0, flat, (out / total).reshape(-1, Hq, d)[rows].to(torch.bfloat16))
            if want_lse:
                lse[b].index_copy_(0, flat, (m + total.log()).reshape(-1, Hq)[rows])
    return (o, lse) if want_lse else o


def _plain_sink_bwd(s):
    c = s["case"]
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    scale = 1.0 / math.sqrt(d)
    dq = torch.empty((B, T, Hq, d), device="cuda")
    dk, dv = torch.zeros((B, T, Hkv, d), device="cuda"), torch.zeros((B, T, Hkv, d), device="cuda")
    dalpha, dbeta = torch.zeros((Hq, d), device="cuda"), torch.zeros((Hq, d), device="cuda")
    for b in range(B):
        for t, q, kb, vb, j, x, y, ks, vs in _sink_parts(s, b):
            at = t.clamp(max=T - 1)
            row = q.shape[:4]
            dO = s["dO"][b][at].float().reshape(q.shape)
            lse = s["lse"][b][at].reshape(row)[..., None]
            D = (dO * s["o"][b][at].float().reshape(q.shape)).sum(-1, keepdim=True)
            p, ps = torch.exp(x - lse), torch.exp(y - lse)
            ds = p * (torch.einsum("nrhgd,nkhd->nrhgk", dO, vb) - D)
            dss = ps * (torch.einsum("nrhgd,khd->nrhgk", dO, vs) - D)
            g = scale * (torch.einsum("nrhgk,nkhd->nrhgd", ds, kb) + torch.einsum("nrhgk,khd->nrhgd", dss, ks))
            g = g.reshape(-1, Hq, d)
            rows = (t < T).reshape(-1)
            flat = t.reshape(-1)[rows]
            dq[b].index_copy_(0, flat, (g * s["alpha"])[rows])
            dalpha += (g[rows] * s["q"][b][flat].float()).sum(0)
            dbeta += g[rows].sum(0)
            to = j.clamp(0, T - 1).reshape(-1)  # keys that are none have zeros
            dk[b].index_add_(0, to, scale * torch.einsum("nrhgk,nrhgd->nkhd", ds, q).reshape(-1, Hkv, d))
            dv[b].index_add_(0, to, torch.einsum("nrhgk,nrhgd->nkhd", p, dO).reshape(-1, Hkv, d))
            dk[b, :ks.shape[0]] += scale * torch.einsum("nrhgk,nrhgd->khd", dss, q)
            dv[b, :ks.shape[0]] += torch.einsum("nrhgk,nrhgd->khd", ps, dO)
    return dq, dk, dv, dalpha, dbeta


def _closure(parent):
    """[B, N, N]: does node j lie on the path to node i (itself included)?"""
    N = parent.shape[1]
    eye = torch.eye(N, device=parent.device)
    reach = eye + (parent[:, :, None] == torch.arange(N, device=parent.device))
    for _ in range(max(1, (N - 1).bit_length())):
        reach = (reach @ reach > 0).float()
    return reach > 0


def _plain_tree(s):
    c = s["case"]
    B, N, Hq, Hkv, d, w, ns = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    on_path = _closure(s["parent"])
    depth = on_path.sum(-1) - 1
    n = s["cache_len"].long()
    pos = n[:, None] + depth  # [B, N]
    L = s["k_cache"].shape[1]
    k, v, kt, vt = (s[x].float() for x in ("k_cache", "v_cache", "k_new", "v_new"))
    j = torch.arange(L, device="cuda")[None, None]
    cached = (j < n[:, None, None]).expand(B, N, L)
    near = cached & ((j > pos[:, :, None] - w) | (j < ns))
    near_t = on_path & ((pos[:, None, :] > pos[:, :, None] - w) | (pos[:, None, :] < ns))
    live = torch.ones((B, N), dtype=torch.bool, device="cuda")
    if s["nodes"] is not None:
        live = torch.arange(N, device="cuda")[None] < s["nodes"][:, None]

    def attend(q, alpha, beta, seen, seen_t, out):
        q = ((q.float() * alpha + beta) / math.sqrt(d)).reshape(B, N, Hkv, -1, d)
        x = torch.einsum("bnhgd,bjhd->bhngj", q, k).masked_fill_(~seen[:, None, :, None], -math.inf)
        y = torch.einsum("bnhgd,bjhd->bhngj", q, kt).masked_fill_(~seen_t[:, None, :, None], -math.inf)
        m = torch.maximum(x.amax(-1), y.amax(-1))[..., None]
        x, y = x.sub_(m).exp_(), y.sub_(m).exp_()
        z = torch.einsum("bhngj,bjhd->bhngd", x, v) + torch.einsum("bhngj,bjhd->bhngd", y, vt)
        z = z / (x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True))
        z = z.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d).to(torch.bfloat16)
        out.copy_(torch.where(live[:, :, None, None], z, out))
        return out

    return (attend(s["q"], s["alpha"], s["beta"], near, near_t, s["o"]),
            attend(s["qc"], s["alpha_c"], s["beta_c"], cached, on_path, s["oc"]))


def _plain_accept(s):
    c = s["case"]
    N = c["N"]
    s["cache_len"].copy_(s["lens"])
    on_path = _closure(s["parent"])
    node = s["node"].long()
    mine = on_path.gather(1, node.clamp(min=0)[:, None, None].expand(-1, 1, N))[:, 0] & (node >= 0)[:, None]  # [B, N]
    count = mine.sum(-1)
    # ancestors come before their descendants, so the path is its nodes in order
    order = torch.where(mine, torch.arange(N, device="cuda")[None], N).sort(-1).values
    path = torch.where(order < N, order, torch.full_like(order, -1)).to(torch.int32)
    b, i = (order < N).nonzero(as_tuple=True)
    at = s["lens"].long()[b] + i
    s["k_cache"][b, at] = s["k_new"][b, order[b, i]]
    s["v_cache"][b, at] = s["v_new"][b, order[b, i]]
    s["cache_len"].add_(count.to(torch.int32))
    return path, s["k_cache"], s["v_cache"], s["cache_len"]


# ---------------------------------------------------------------------------------- one pass


def _own(s):
    import long_context_attention_orthros_gb300 as orth

    c, op = s["case"], s["case"]["op"]
    if op == "sink_fwd":
        return orth.swa_sink_fwd(s["q"], s["k"], s["v"], s["alpha"], s["beta"], c["sinks"], window=c["window"],
                                 lse=True if c["lse"] else None)
    if op == "sink_bwd":
        if "workspace" not in s:
            n = orth.swa_sink_bwd_workspace_size(c["B"], c["T"], c["Hq"], c["Hkv"], c["d"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return orth.swa_sink_bwd(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["o"], s["dO"], s["lse"], c["sinks"],
                                 window=c["window"], workspace=s["workspace"])
    if op == "accept":
        s["cache_len"].copy_(s["lens"])
        path = orth.decode_tree_accept(s["k_new"], s["v_new"], s["parent"], s["node"], s["k_cache"], s["v_cache"],
                                       s["cache_len"])
        return path, s["k_cache"], s["v_cache"], s["cache_len"]
    if "workspace" not in s:
        n = orth.decode_tree_workspace_size(c["B"], c["N"], s["k_cache"].shape[1], c["Hq"], c["Hkv"], c["d"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return orth.decode_tree(s["q"], s["qc"], s["k_new"], s["v_new"], s["parent"], s["k_cache"], s["v_cache"],
                            s["cache_len"], s["alpha"], s["beta"], s["alpha_c"], s["beta_c"], window=c["window"],
                            sinks=c["sinks"], nodes=s["nodes"], o=s["o"], oc=s["oc"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "sink_fwd":
        return _plain_sink_fwd(state, state["case"]["lse"])
    return {"sink_bwd": _plain_sink_bwd, "tree": _plain_tree, "accept": _plain_accept}[op](state)


# ---------------------------------------------------------------------------------- accounting


def work(case):
    """Bytes: each input once, each output once.  A ragged batch counts its mean lengths (half the
    longest, but for the first sequence); a tree's paths count half its nodes."""
    c, op = case, case["op"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    if op in ("sink_fwd", "sink_bwd"):
        T = c["T"]
        w, ns = min(c["window"], T), min(c["sinks"], T)
        far = T - w  # rows that have left the first key behind: they see up to ns sinks beside the window
        m = min(ns, far)
        keys = w * (w + 1) // 2 + far * w + m * (m + 1) // 2 + (far - m) * ns
        if op == "sink_fwd":
            return {"bytes": 4 * B * T * (Hq + Hkv) * d + 8 * Hq * d + (4 * B * T * Hq if c["lse"] else 0),
                    "flops": 4 * d * Hq * B * keys}
        return {"bytes": B * T * (Hq * d * (3 * 2 + 4) + Hkv * d * (2 * 2 + 2 * 4) + 4 * Hq) + 16 * Hq * d,
                "flops": 10 * d * Hq * B * keys}
    N = c["N"]
    if op == "accept":  # half a chain's rows, or a path of a few, moved; the trees and the paths
        moved = B * (N / 2 if c["shape"] == "chain" else math.log2(N + 1))
        return {"bytes": 8 * moved * Hkv * d + 8 * B * N + 12 * B, "flops": 0}
    mean = (1 + (B - 1) / 2) if c["ragged"] else B  # sequences of full length that it amounts to
    rows, nodes = mean * c["L"], mean * N
    pairs = N * c["L"] * ((1 + (B - 1) / 4) if c["ragged"] else B) + nodes * (min(c["window"], c["L"]) + c["sinks"])
    return {"bytes": 4 * (rows + nodes) * Hkv * d + 8 * nodes * Hq * d + 16 * Hq * d + 4 * B * N + 4 * B,
            "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------------------------- exact values


def _exact_row_blocks(s, b, h, block=512):
    """Blocks of rows of one head in 64 bits: rows, queries, the keys' rows, weights' logits (masked)."""
    c = s["case"]
    T, G = c["T"], c["Hq"] // c["Hkv"]
    k, v = s["k"][b, :, h // G].double(), s["v"][b, :, h // G].double()
    q = s["q"][b, :, h].double() * s["alpha"][h].double() + s["beta"][h].double()
    for t0 in range(0, T, block):
        t = torch.arange(t0, min(T, t0 + block), device="cuda")
        lo = max(0, t0 - c["window"] + 1)
        ns = min(c["sinks"], lo)
        j = torch.cat([torch.arange(ns, device="cuda"), torch.arange(lo, int(t[-1]) + 1, device="cuda")])
        x = q[t] @ k[j].T / math.sqrt(c["d"])
        seen = (j[None] <= t[:, None]) & ((j[None] > t[:, None] - c["window"]) | (j[None] < c["sinks"]))
        yield t, q[t], j, k[j], v[j], torch.where(seen, x, torch.full_like(x, -math.inf))


def exact(case, seed):
    c, op = case, case["op"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    if op == "accept":
        s = prepare(case, seed)
        k, v = s["k_cache"].double(), s["v_cache"].double()
        parent, lens, node = s["parent"].tolist(), s["lens"].tolist(), s["node"].tolist()
        for b in range(B):
            path, i = [], node[b]
            while i >= 0:
                path.insert(0, i)
                i = parent[b][i]
            for a, i in enumerate(path):
                k[b, lens[b] + a], v[b, lens[b] + a] = s["k_new"][b, i].double(), s["v_new"][b, i].double()
        return None, k, v, None
    if op in ("sink_fwd", "sink_bwd"):
        T = c["T"]
        if B * Hq * (T // 512 + 1) * (min(c["window"], T) + 512) * 512 * d > 3e12 or B * Hq * (T // 512 + 1) > 40000:
            return None
        s = prepare(case, seed)
        f64 = dict(dtype=torch.float64, device="cuda")
        o, lse = torch.empty((B, T, Hq, d), **f64), torch.empty((B, T, Hq), **f64)
        dq, dk, dv = (torch.zeros((B, T, n, d), **f64) for n in (Hq, Hkv, Hkv))
        da, db = torch.zeros((Hq, d), **f64), torch.zeros((Hq, d), **f64)
        for b in range(B):
            for h in range(Hq):
                for t, q, j, k, v, x in _exact_row_blocks(s, b, h):
                    if op == "sink_fwd":
                        m = torch.logsumexp(x, -1)
                        lse[b, t, h] = m
                        o[b, t, h] = torch.exp(x - m[:, None]) @ v
                        continue
                    p = torch.exp(x - s["lse"][b, t, h].double()[:, None])
                    dO = s["dO"][b, t, h].double()
                    ds = p * (dO @ v.T - (dO * s["o"][b, t, h].double()).sum(-1, keepdim=True)) / math.sqrt(d)
                    g = ds @ k
                    dq[b, t, h] = g * s["alpha"][h].double()
                    da[h] += (g * s["q"][b, t, h].double()).sum(0)
                    db[h] += g.sum(0)
                    dk[b, :, h // (Hq // Hkv)].index_add_(0, j, ds.T @ q)
                    dv[b, :, h // (Hq // Hkv)].index_add_(0, j, p.T @ dO)
        if op == "sink_bwd":
            return dq, dk, dv, da, db
        return (o, lse) if c["lse"] else o
    s = prepare(case, seed)
    o, oc = s["o"].double(), s["oc"].double()
    parent, lens = s["parent"].tolist(), s["cache_len"].tolist()
    nodes = [c["N"]] * B if s["nodes"] is None else s["nodes"].tolist()
    G = Hq // Hkv
    for b in range(B):
        k = torch.cat([s["k_cache"][b, :lens[b]], s["k_new"][b]]).double()
        v = torch.cat([s["v_cache"][b, :lens[b]], s["v_new"][b]]).double()
        place = list(range(lens[b]))  # position of each row, the drafted ones' behind
        paths = []
        for i in range(c["N"]):
            up = parent[b][i]
            paths.append((paths[up] if up >= 0 else []) + [i])
            place.append(lens[b] + len(paths[i]) - 1)
        place = torch.tensor(place, device="cuda")
        n = nodes[b]
        if n == 0:
            continue
        whole = torch.zeros((n, len(place)), dtype=torch.bool, device="cuda")
        whole[:, :lens[b]] = True
        for i in range(n):
            whole[i, torch.tensor(paths[i], device="cuda") + lens[b]] = True
        at = place[lens[b]:lens[b] + n, None]
        near = whole & ((place[None] > at - c["window"]) | (place[None] < c["sinks"]))
        for out, x, al, be, seen in ((o, "q", "alpha", "beta", near), (oc, "qc", "alpha_c", "beta_c", whole)):
            for h in range(Hq):
                q = s[x][b, :n, h].double() * s[al][h].double() + s[be][h].double()
                y = q @ k[:, h // G].T / math.sqrt(d)
                out[b, :n, h] = torch.softmax(torch.where(seen, y, torch.full_like(y, -math.inf)), -1) @ v[:, h // G]
    return o, oc
