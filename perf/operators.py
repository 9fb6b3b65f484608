"""Serving operators over an 8-bit KV cache and over a shared prompt prefix: the cases that are
measured, their plain forms, and the calls a user makes.

* ``quantize`` / ``dequantize``: a prompt's K and V rows written into an 8-bit cache (e4m3 or
  int8 codes, one power-of-two exponent for each row of each KV head) and read back as bf16;
* ``decode_q8``: one decode step over such a cache (append, window attention of the new base
  token, attention of its output copy over the whole cache);
* ``decode_prefix``: one decode step for a batch whose sequences share one prompt prefix;
* ``xattn_prefix``: output copies of a batch over the shared prefix and their own rows.

A row's exponent e is the smallest whole number for which every |x| 2^-e of the row is at most
the code's largest value (448 for e4m3, 127 for int8; 0 for a row of zeros), the codes are
x 2^-e rounded to nearest even, and they stand for code 2^e.
"""
import math

import torch

own = False

_HEADS = ((2, 1, 64), (8, 2, 64), (4, 4, 64), (16, 1, 128), (8, 4, 128), (32, 8, 128))


def listed():
    q = {"Hq": 32, "Hkv": 8, "d": 128, "window": 128}
    s = {"Hq": 8, "Hkv": 2, "d": 64, "window": 128}
    return [
        # a 128K prompt of two sequences goes into the cache of the 8B-class layer
        {"name": "quantize prompt 2x131072 e4m3", "op": "quantize", "B": 2, "T": 131072, "Hkv": 8, "d": 128,
         "code": "e4m3", "ragged": False},
        # a short chunk of a padded batch, small heads
        {"name": "quantize chunk 4x513 int8", "op": "quantize", "B": 4, "T": 513, "Hkv": 2, "d": 64,
         "code": "int8", "ragged": True},
        # the cache of a 16K prompt read back for another pass over it
        {"name": "dequantize 2x16384 e4m3", "op": "dequantize", "B": 2, "T": 16384, "Hkv": 8, "d": 128,
         "code": "e4m3", "ragged": False},
        # the window in front of the next chunk of a prompt, read back
        {"name": "dequantize window 8x128 int8", "op": "dequantize", "B": 8, "T": 128, "Hkv": 8, "d": 128,
         "code": "int8", "ragged": True},
        # decode behind a 128K prompt, batch 2
        {"name": "decode q8 2x131072 e4m3", "op": "decode_q8", "B": 2, "L": 131072, "code": "e4m3",
         "ragged": False, **q},
        # a batch of sequences of every length up to 16K
        {"name": "decode q8 ragged 8x16384 int8", "op": "decode_q8", "B": 8, "L": 16384, "code": "int8",
         "ragged": True, **q},
        # the first tokens behind a short prompt: latency counts
        {"name": "decode q8 1x300 e4m3", "op": "decode_q8", "B": 1, "L": 300, "code": "e4m3",
         "ragged": False, **s},
        # eight answers sampled from one 128K prompt
        {"name": "decode prefix 8 over 131072", "op": "decode_prefix", "B": 8, "P": 131072, "L": 1000,
         "ragged": True, **q},
        # many users behind one system prompt
        {"name": "decode prefix 64 over 16384", "op": "decode_prefix", "B": 64, "P": 16384, "L": 500,
         "ragged": True, **q},
        # a few short answers from a short prompt: latency counts
        {"name": "decode prefix 4 over 511", "op": "decode_prefix", "B": 4, "P": 511, "L": 70,
         "ragged": True, **s},
        # the last prompt position of eight user turns behind one long prefix
        {"name": "xattn prefix 8x1 over 32768", "op": "xattn_prefix", "B": 8, "T_out": 1, "P": 32768, "T": 500,
         "Hq": 32, "Hkv": 8, "d": 128},
        # answer spans of four samples of one prompt (a training rollout)
        {"name": "xattn prefix 4x256 over 16384", "op": "xattn_prefix", "B": 4, "T_out": 256, "P": 16384,
         "T": 1000, "Hq": 32, "Hkv": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "decode_q8", "decode_prefix", "xattn_prefix"])
    Hq, Hkv, d = rng.choice(_HEADS)
    code = rng.choice(["e4m3", "int8"])
    window = rng.choice([1, 77, 128, 128, 128, 300])
    budget = 1 << 27  # values of K (and of V) that a case holds
    if op in ("quantize", "dequantize"):
        B = _log(rng, 1, 16)
        T = _log(rng, 1, min(131072, budget // (B * Hkv * d)))
        return {"op": op, "B": B, "T": T, "Hkv": Hkv, "d": d, "code": code, "ragged": rng.random() < 0.5}
    if op == "decode_q8":
        B = _log(rng, 1, 32)
        L = _log(rng, 1, min(131072, budget // (B * Hkv * d)))
        return {"op": op, "B": B, "L": L, "code": code, "ragged": rng.random() < 0.6, "Hq": Hq, "Hkv": Hkv,
                "d": d, "window": window}
    P = _log(rng, 1, min(131072, budget // (Hkv * d)))
    if op == "decode_prefix":
        B = _log(rng, 1, max(1, min(64, (1 << 28) // (P * Hq))))
        return {"op": op, "B": B, "P": P, "L": _log(rng, 1, 2000), "ragged": rng.random() < 0.6, "Hq": Hq,
                "Hkv": Hkv, "d": d, "window": window}
    B = _log(rng, 1, max(1, min(16, (1 << 28) // (P * Hq))))
    T_out = _log(rng, 1, max(1, min(512, (1 << 28) // (P * Hq * B))))
    return {"op": op, "B": B, "T_out": T_out, "P": P, "T": _log(rng, 1, 2000), "Hq": Hq, "Hkv": Hkv, "d": d}


# ---------------------------------------------------------------------------------- inputs


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _lens(gen, B, L, ragged):
    if not ragged:
        return torch.full((B,), L, dtype=torch.int32, device="cuda")
    n = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = L  # the longest fills the range
    return n


def _vectors(gen, Hq, d):
    one = torch.ones((Hq, d), device="cuda")
    return {"alpha": one + 0.1 * _normal(gen, Hq, d, dtype=torch.float32),
            "beta": 0.1 * _normal(gen, Hq, d, dtype=torch.float32),
            "alpha_c": one + 0.1 * _normal(gen, Hq, d, dtype=torch.float32),
            "beta_c": 0.1 * _normal(gen, Hq, d, dtype=torch.float32)}


def _cache(gen, B, L_max, Hkv, d, code):
    """An 8-bit cache in use: every row holds some token's codes."""
    c, e = _plain_codes(_normal(gen, B, L_max, Hkv, d), code)
    return c, e.permute(0, 2, 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, op = case, case["op"]
    s = {"case": dict(c)}
    if op in ("quantize", "dequantize"):
        B, T, Hkv, d = c["B"], c["T"], c["Hkv"], c["d"]
        front = 16 if c["ragged"] else 0  # rows that the cache holds already
        L_max = (front + T + 127) // 128 * 128
        s["start"] = torch.randint(0, front + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["rows"] = _lens(gen, B, T, c["ragged"])
        s["k8"], s["k_exp"] = _cache(gen, B, L_max, Hkv, d, c["code"])
        s["v8"], s["v_exp"] = _cache(gen, B, L_max, Hkv, d, c["code"])
        s["k"], s["v"] = _normal(gen, B, T, Hkv, d), _normal(gen, B, T, Hkv, d)
        return s
    Hq, Hkv, d, B = c["Hq"], c["Hkv"], c["d"], c["B"]
    s.update(_vectors(gen, Hq, d))
    if op == "xattn_prefix":
        s["qc"] = _normal(gen, B, c["T_out"], Hq, d)
        s["pos"] = torch.randint(0, c["T"], (B, c["T_out"]), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"][0, 0] = c["T"] - 1
        s["k"], s["v"] = _normal(gen, B, c["T"], Hkv, d), _normal(gen, B, c["T"], Hkv, d)
        s["kp"], s["vp"] = _normal(gen, c["P"], Hkv, d), _normal(gen, c["P"], Hkv, d)
        return s
    s["q"], s["qc"] = _normal(gen, B, Hq, d), _normal(gen, B, Hq, d)
    s["k_new"], s["v_new"] = _normal(gen, B, Hkv, d), _normal(gen, B, Hkv, d)
    s["lens"] = _lens(gen, B, c["L"], c["ragged"])  # what the scheduler knows of each sequence
    s["cache_len"] = s["lens"].clone()
    L_max = (c["L"] + 128) // 128 * 128
    if op == "decode_q8":
        s["k8"], s["k_exp"] = _cache(gen, B, L_max, Hkv, d, c["code"])
        s["v8"], s["v_exp"] = _cache(gen, B, L_max, Hkv, d, c["code"])
    else:
        s["k_cache"], s["v_cache"] = _normal(gen, B, L_max, Hkv, d), _normal(gen, B, L_max, Hkv, d)
        s["kp"], s["vp"] = _normal(gen, c["P"], Hkv, d), _normal(gen, c["P"], Hkv, d)
    return s


# ---------------------------------------------------------------------------------- plain forms


def _pow2(e):
    """2^e as fp32, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_codes(x, code):
    """Rows [..., d] as codes and exponents int8 [...]."""
    x = x.float()
    most, top = (448.0, 8) if code == "e4m3" else (127.0, 6)
    amax = x.abs().amax(-1)
    mant, ex = torch.frexp(amax)  # amax = mant 2^ex, mant in [0.5, 1)
    e = ex.to(torch.int32) - 1 - top
    e = torch.where(mant * 2.0 ** (top + 1) > most, e + 1, e)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-126, 127)
    y = x * _pow2(-e)[..., None]
    c = y.to(torch.float8_e4m3fn) if code == "e4m3" else torch.round(y).to(torch.int8)
    return c, e.to(torch.int8)


def _plain_values(c, e):
    """Codes [B, L, Hkv, d] and exponents [B, Hkv, L] as fp32 values."""
    return c.float() * _pow2(e.permute(0, 2, 1))[..., None]


def _set_rows(cache, at, rows, keep=None):
    """cache[b, at[b, t]] = rows[b, t] (where keep), in place; at [B, T] of distinct rows."""
    raw = cache.view(torch.uint8) if cache.dtype in (torch.float8_e4m3fn, torch.int8) else cache
    new = rows.view(raw.dtype) if raw.dtype == torch.uint8 else rows
    index = at.long().reshape(at.shape + (1,) * (raw.dim() - 2)).expand(new.shape)
    if keep is not None:
        new = torch.where(keep.reshape(keep.shape + (1,) * (raw.dim() - 2)), new, raw.gather(1, index))
    raw.scatter_(1, index, new)


def _plain_quantize(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda", dtype=torch.int32)[None]
    at, keep = s["start"][:, None] + t, t < s["rows"][:, None]
    ck, ek = _plain_codes(s["k"], c["code"])
    cv, ev = _plain_codes(s["v"], c["code"])
    _set_rows(s["k8"], at, ck, keep)
    _set_rows(s["v8"], at, cv, keep)
    _set_rows(s["k_exp"].transpose(1, 2), at, ek, keep)
    _set_rows(s["v_exp"].transpose(1, 2), at, ev, keep)
    return s["k8"], s["v8"], s["k_exp"], s["v_exp"]


def _plain_dequantize(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda", dtype=torch.int32)[None]
    at, keep = (s["start"][:, None] + t).long(), (t < s["rows"][:, None])[:, :, None, None]
    index = at[:, :, None, None].expand(c["B"], c["T"], c["Hkv"], c["d"])
    ie = at[:, None, :].expand(c["B"], c["Hkv"], c["T"])
    ck = s["k8"].view(torch.uint8).gather(1, index).view(s["k8"].dtype)
    cv = s["v8"].view(torch.uint8).gather(1, index).view(s["v8"].dtype)
    k = _plain_values(ck, s["k_exp"].gather(2, ie)).to(torch.bfloat16)
    v = _plain_values(cv, s["v_exp"].gather(2, ie)).to(torch.bfloat16)
    s["k"].copy_(torch.where(keep, k, s["k"]))  # rows behind a sequence's last stay as they were
    s["v"].copy_(torch.where(keep, v, s["v"]))
    return s["k"], s["v"]


def _weights(x, seen):
    """exp(x - max) over the keys that are seen, and its sum."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    w = torch.exp(x - x.amax(-1, keepdim=True))
    return w, w.sum(-1, keepdim=True)


def _grouped(q, alpha, beta, Hkv):
    """Scale-offset queries [..., Hq, d] as fp32 [..., Hkv, G, d], with the softmax scale."""
    d = q.shape[-1]
    q = (q.float() * alpha + beta) / math.sqrt(d)
    return q.reshape(q.shape[:-2] + (Hkv, -1, d))


def _plain_decode_q8(s):
    c = s["case"]
    s["cache_len"].copy_(s["lens"])
    at = s["cache_len"][:, None]
    ck, ek = _plain_codes(s["k_new"], c["code"])
    cv, ev = _plain_codes(s["v_new"], c["code"])
    _set_rows(s["k8"], at, ck[:, None])
    _set_rows(s["v8"], at, cv[:, None])
    _set_rows(s["k_exp"].transpose(1, 2), at, ek[:, None])
    _set_rows(s["v_exp"].transpose(1, 2), at, ev[:, None])
    k, v = _plain_values(s["k8"], s["k_exp"]), _plain_values(s["v8"], s["v_exp"])
    j = torch.arange(k.shape[1], device="cuda")[None, None, None]
    p = s["cache_len"].long()[:, None, None, None]

    def attend(q, lo):
        x = torch.einsum("bhgd,bjhd->bhgj", q, k)
        w, total = _weights(x, (j <= p) & (j >= lo))
        return (torch.einsum("bhgj,bjhd->bhgd", w, v) / total).reshape(c["B"], c["Hq"], c["d"]).to(torch.bfloat16)

    o = attend(_grouped(s["q"], s["alpha"], s["beta"], c["Hkv"]), p - c["window"] + 1)
    oc = attend(_grouped(s["qc"], s["alpha_c"], s["beta_c"], c["Hkv"]), torch.zeros_like(p))
    s["cache_len"].add_(1)
    return o, oc, s["k8"], s["v8"], s["k_exp"], s["v_exp"], s["cache_len"]


def _plain_decode_prefix(s):
    c, P = s["case"], s["case"]["P"]
    s["cache_len"].copy_(s["lens"])
    _set_rows(s["k_cache"], s["cache_len"][:, None], s["k_new"][:, None])
    _set_rows(s["v_cache"], s["cache_len"][:, None], s["v_new"][:, None])
    k, v, kp, vp = (s[n].float() for n in ("k_cache", "v_cache", "kp", "vp"))
    j = torch.arange(P + k.shape[1], device="cuda")[None, None, None]
    p = P + s["cache_len"].long()[:, None, None, None]

    def attend(q, lo):
        x = torch.cat([torch.einsum("bhgd,jhd->bhgj", q, kp), torch.einsum("bhgd,bjhd->bhgj", q, k)], -1)
        w, total = _weights(x, (j <= p) & (j >= lo))
        y = torch.einsum("bhgj,jhd->bhgd", w[..., :P], vp) + torch.einsum("bhgj,bjhd->bhgd", w[..., P:], v)
        return (y / total).reshape(c["B"], c["Hq"], c["d"]).to(torch.bfloat16)

    o = attend(_grouped(s["q"], s["alpha"], s["beta"], c["Hkv"]), p - c["window"] + 1)
    oc = attend(_grouped(s["qc"], s["alpha_c"], s["beta_c"], c["Hkv"]), torch.zeros_like(p))
    s["cache_len"].add_(1)
    return o, oc, s["k_cache"], s["v_cache"], s["cache_len"]


def _plain_xattn_prefix(s):
    c, P = s["case"], s["case"]["P"]
    k, v, kp, vp = (s[n].float() for n in ("k", "v", "kp", "vp"))
    q = _grouped(s["qc"], s["alpha_c"], s["beta_c"], c["Hkv"])  # [B, T_out, Hkv, G, d]
    x = torch.cat([torch.einsum("bihgd,jhd->bhigj", q, kp), torch.einsum("bihgd,bjhd->bhigj", q, k)], -1)
    j = torch.arange(P + c["T"], device="cuda")
    w, total = _weights(x, j <= P + s["pos"].long()[:, None, :, None, None])
    y = torch.einsum("bhigj,jhd->bhigd", w[..., :P], vp) + torch.einsum("bhigj,bjhd->bhigd", w[..., P:], v)
    return (y / total).permute(0, 2, 1, 3, 4).reshape(c["B"], c["T_out"], c["Hq"], c["d"]).to(torch.bfloat16)


# ---------------------------------------------------------------------------------- one pass


def _own(s):
    import long_context_attention_orthros_gb300 as orth

    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        orth.kv_quantize(s["k"], s["v"], s["k8"], s["v8"], s["k_exp"], s["v_exp"], start=s["start"], rows=s["rows"])
        return s["k8"], s["v8"], s["k_exp"], s["v_exp"]
    if op == "dequantize":
        orth.kv_dequantize(s["k8"], s["v8"], s["k_exp"], s["v_exp"], s["k"], s["v"], start=s["start"], rows=s["rows"])
        return s["k"], s["v"]
    if op == "xattn_prefix":
        if "workspace" not in s:
            n = orth.xattn_prefix_workspace_size(c["B"], c["T_out"], c["P"], c["T"], c["Hq"], c["Hkv"], c["d"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return orth.xattn_prefix_fwd(s["qc"], s["pos"], s["kp"], s["vp"], s["k"], s["v"], s["alpha_c"], s["beta_c"],
                                     workspace=s["workspace"])
    vectors = (s["alpha"], s["beta"], s["alpha_c"], s["beta_c"])
    s["cache_len"].copy_(s["lens"])
    if op == "decode_q8":
        if "workspace" not in s:
            n = orth.decode_q8_workspace_size(c["B"], s["k8"].shape[1], c["Hq"], c["Hkv"], c["d"])
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        o, oc = orth.decode_step_q8(s["q"], s["qc"], s["k_new"], s["v_new"], s["k8"], s["v8"], s["k_exp"], s["v_exp"],
                                    s["cache_len"], *vectors, window=c["window"], workspace=s["workspace"])
        return o, oc, s["k8"], s["v8"], s["k_exp"], s["v_exp"], s["cache_len"]
    if "workspace" not in s:
        n = orth.decode_prefix_workspace_size(c["B"], c["P"], s["k_cache"].shape[1], c["Hq"], c["Hkv"], c["d"])
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    o, oc = orth.decode_step_prefix(s["q"], s["qc"], s["k_new"], s["v_new"], s["kp"], s["vp"], s["k_cache"],
                                    s["v_cache"], s["cache_len"], *vectors, window=c["window"],
                                    workspace=s["workspace"])
    return o, oc, s["k_cache"], s["v_cache"], s["cache_len"]


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "dequantize": _plain_dequantize, "decode_q8": _plain_decode_q8,
            "decode_prefix": _plain_decode_prefix, "xattn_prefix": _plain_xattn_prefix}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------- accounting


def work(case):
    """Bytes: each input once, each output once.  A ragged batch counts its mean length (half the
    longest, but for the first sequence)."""
    c, op = case, case["op"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]

    def rows(n):
        return n + (B - 1) * n / 2 if c["ragged"] else B * n

    if op in ("quantize", "dequantize"):
        n = rows(c["T"]) * Hkv * 2
        return {"bytes": n * (2 * d + d + 1), "flops": n * d * 2}
    Hq = c["Hq"]
    if op == "xattn_prefix":
        R = B * c["T_out"]
        keys = c["P"] + (c["T"] + 1) / 2  # a copy's mean number of keys
        return {"bytes": 4 * R * Hq * d + 4 * (c["P"] + B * c["T"]) * Hkv * d + 8 * Hq * d + 4 * R,
                "flops": 4 * d * Hq * R * keys}
    n = rows(c["L"])
    small = 8 * B * Hq * d + 16 * Hq * d + 4 * B * Hkv * d + 8 * B  # q, o of both streams, vectors, new rows
    if op == "decode_q8":
        return {"bytes": small + 2 * (n + B) * Hkv * (d + 1), "flops": 4 * d * Hq * (n + B * min(c["window"], c["L"] + 1))}
    return {"bytes": small + 4 * (n + B) * Hkv * d + 4 * c["P"] * Hkv * d,
            "flops": 4 * d * Hq * (n + B * c["P"] + B * min(c["window"], c["P"]))}


# ---------------------------------------------------------------------------------- exact values


def _exact_codes(x, code):
    """The definition in 64 bits: exponents by comparison, codes by rounding to the code's grid."""
    x = x.double()
    most = 448.0 if code == "e4m3" else 127.0
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(amax, -126.0)
    for n in range(7, -1, -1):  # the largest whole number that still overflows, by bisection
        up = torch.exp2(torch.tensor(float(n), dtype=torch.float64, device=x.device))
        e = torch.where(amax * torch.exp2(-(e + up - 1)) > most, e + up, e)
    e = torch.where(amax > 0, e.clamp(max=127), torch.zeros_like(e))
    y = x * torch.exp2(-e)
    if code == "e4m3":
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step
    else:
        y = torch.round(y)
    return y, e[..., 0]


def _exact_rows(q, parts):
    """softmax attention of q [R, d] over the keys of several (k [n, d], v [n, d], seen [R, n])."""
    x = [torch.where(m, q @ k.T, torch.full((), -math.inf, dtype=torch.float64, device=q.device)) for k, _, m in parts]
    top = torch.stack([y.amax(-1) for y in x if y.shape[1]]).amax(0)[:, None]
    w = [torch.exp(y - top) for y in x]
    return sum(a @ v for a, (_, v, _) in zip(w, parts)) / sum(a.sum(-1, keepdim=True) for a in w)


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if op == "quantize":
        out = {}
        for n in ("k", "v"):
            y, _ = _exact_codes(s[n], c["code"])
            out[n] = s[n + "8"].double()
            for b in range(B):
                st, nr = int(s["start"][b]), int(s["rows"][b])
                out[n][b, st:st + nr] = y[b, :nr]
            del y
        return out["k"], out["v"], None, None
    if op == "dequantize":
        out = {}
        for n in ("k", "v"):
            out[n] = s[n].double()
            for b in range(B):
                st, nr = int(s["start"][b]), int(s["rows"][b])
                e = s[n + "_exp"][b, :, st:st + nr].T.double()[..., None]
                out[n][b, :nr] = s[n + "8"][b, st:st + nr].double() * torch.exp2(e)
        return out["k"], out["v"]
    Hq, G, scale = c["Hq"], c["Hq"] // Hkv, d ** -0.5

    def query(q, al, be):
        return (q.double() * s[al].double() + s[be].double()) * scale

    if op == "xattn_prefix":
        o = torch.empty((B, c["T_out"], Hq, d), dtype=torch.float64, device="cuda")
        q = query(s["qc"], "alpha_c", "beta_c")
        j = torch.arange(c["T"], device="cuda")[None]
        for h in range(Hkv):
            kp, vp = s["kp"][:, h].double(), s["vp"][:, h].double()
            for b in range(B):
                rows = q[b, :, h * G:(h + 1) * G].reshape(-1, d)
                seen = j <= s["pos"][b].repeat_interleave(G)[:, None]
                every = torch.ones((1, c["P"]), dtype=torch.bool, device="cuda")
                y = _exact_rows(rows, [(kp, vp, every), (s["k"][b, :, h].double(), s["v"][b, :, h].double(), seen)])
                o[b, :, h * G:(h + 1) * G] = y.reshape(c["T_out"], G, d)
        return o
    o, oc = (torch.empty((B, Hq, d), dtype=torch.float64, device="cuda") for _ in range(2))
    q, qc = query(s["q"], "alpha", "beta"), query(s["qc"], "alpha_c", "beta_c")
    if op == "decode_q8":
        (kn, ken), (vn, ven) = _exact_codes(s["k_new"], c["code"]), _exact_codes(s["v_new"], c["code"])
        kn, vn = kn * torch.exp2(ken)[..., None], vn * torch.exp2(ven)[..., None]
    else:
        kn, vn = s["k_new"].double(), s["v_new"].double()
    for b in range(B):
        n = int(s["lens"][b])
        for h in range(Hkv):
            if op == "decode_q8":
                k = s["k8"][b, :n, h].double() * torch.exp2(s["k_exp"][b, h, :n].double())[:, None]
                v = s["v8"][b, :n, h].double() * torch.exp2(s["v_exp"][b, h, :n].double())[:, None]
            else:
                k = torch.cat([s["kp"][:, h], s["k_cache"][b, :n, h]]).double()
                v = torch.cat([s["vp"][:, h], s["v_cache"][b, :n, h]]).double()
            k, v = torch.cat([k, kn[b, h][None]]), torch.cat([v, vn[b, h][None]])
            for y, rows, first in ((o, q, max(0, len(k) - c["window"])), (oc, qc, 0)):
                r = slice(h * G, (h + 1) * G)
                every = torch.ones((1, 1), dtype=torch.bool, device="cuda")
                y[b, r] = _exact_rows(rows[b, r], [(k[first:], v[first:], every)])
    return (o, oc, None, None, None, None, None) if op == "decode_q8" else (o, oc, None, None, None)
