"""GPU tests of the 8-bit KV cache: writing prompt rows, reading them back, and the decode step over such a
cache, against the numpy definition and the fp64 oracle.  The values codes stand for are exact in bf16, so the
oracle's bf16 decode step over them is the decode step over the codes."""
import math

import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
import oracle
from synthetic import DecodeConfig, make_decode, normal_bf16
from tests.gpu_util import assert_parity, bf, bits, dev, f32, i32, val
from tests.q8_util import quantize, value_bits

pytestmark = pytest.mark.gpu

DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
NAN_CODE, ANY_EXP = 0x7F, 127  # what rows without a token hold in these tests


def codes(x: np.ndarray, code: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x).view(np.int8)).to(dev()).view(DTYPE[code])


def raw(t: torch.Tensor) -> np.ndarray:
    return t.view(torch.int8).cpu().numpy().view(np.uint8)


def exps(e: np.ndarray) -> torch.Tensor:
    """[B, L, Hkv] numpy exponents -> [B, Hkv, L] on the device."""
    return torch.from_numpy(np.ascontiguousarray(e.transpose(0, 2, 1))).to(dev())


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=dev())


# ------------------------------------------------------------------------------ write and read back


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("B,T,Hkv,d,L_max,start,rows", [
    (1, 1, 1, 64, 16, None, None),
    (2, 33, 2, 128, 48, (0, 15), None),
    (3, 40, 3, 64, 96, (7, 0, 56), (0, 1, 40)),    # nothing, one row, all rows up to the end of the cache
    (2, 129, 8, 128, 160, (31, 1), (128, 127)),
    (1, 70, 67, 64, 80, (3,), (65,)),               # more heads than one block takes
])
def test_quantize_and_read_back(code, B, T, Hkv, d, L_max, start, rows):
    k, v = (normal_bf16(70 + T, n, (B, T, Hkv, d)) for n in ("k", "v"))
    k[:, 0, 0] = 0                       # a row of zeros
    v[:, T // 2] = np.uint16(0x0040)     # subnormal values: below the exponents' range
    k[0, T - 1, 0, :7] = np.uint16(0xC7FF)
    ck, ek = quantize(k, code)
    cv, ev = quantize(v, code)
    want = [np.full((B, L_max, Hkv, d), NAN_CODE, np.uint8) for _ in range(2)]
    want_e = [np.full((B, L_max, Hkv), ANY_EXP, np.int8) for _ in range(2)]
    k8, v8 = (codes(w, code) for w in want)
    ke, ve = (exps(w) for w in want_e)
    for b in range(B):
        s, n = (start[b] if start else 0), (rows[b] if rows else T)
        want[0][b, s:s + n], want[1][b, s:s + n] = ck[b, :n], cv[b, :n]
        want_e[0][b, s:s + n], want_e[1][b, s:s + n] = ek[b, :n], ev[b, :n]
    st, nr = (None if x is None else i32(np.array(x)) for x in (start, rows))
    err = error_word()
    orth.kv_quantize(bf(k), bf(v), k8, v8, ke, ve, start=st, rows=nr, dev_err=err)
    back = [torch.full((B, T, Hkv, d), 7.0, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    orth.kv_dequantize(k8, v8, ke, ve, *back, start=st, rows=nr, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for got, w in ((k8, want[0]), (v8, want[1])):
        np.testing.assert_array_equal(raw(got), w)
    for got, w in ((ke, want_e[0]), (ve, want_e[1])):
        np.testing.assert_array_equal(got.cpu().numpy(), w.transpose(0, 2, 1))
    for got, c, e in ((back[0], ck, ek), (back[1], cv, ev)):
        for b in range(B):
            n = rows[b] if rows else T
            exact = np.float64(1) * e[b, :n] > -120  # codes of deeper rows can fall below bf16's smallest
            g, w = bits(got)[b], None
            for r in range(n):
                for h in range(Hkv):
                    if exact[r, h]:
                        w = value_bits(c[b, r, h], e[b, r, h], code)
                        np.testing.assert_array_equal(g[r, h], w)
            assert (g[n:] == 0x40E0).all()  # 7.0: left as it was


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_values_that_are_not_finite(code):
    x = normal_bf16(5, "k", (1, 2, 1, 64))
    x[0, 0, 0, 3], x[0, 0, 0, 4], x[0, 0, 0, 5] = 0x7F80, 0xFF80, 0x7FC0  # inf, -inf, NaN
    fine = x.copy()
    fine[0, 0, 0, 3:6] = 0
    c, e = quantize(fine, code)
    c[0, 0, 0, 3:6] = (0x7F, 0x7F, 0x7F) if code == "e4m3" else (127, 256 - 127, 0)
    cache = orth.kv_cache_q8(1, 2, 1, 64, dev(), dtype=DTYPE[code])
    err = error_word()
    orth.kv_quantize(bf(x), bf(fine), *cache, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == orth.DEVERR_RANGE
    got = raw(cache[0])[0, :2, 0]
    if code == "e4m3":
        assert (got[0, 3:6] & 0x7F == 0x7F).all()  # NaN of either sign
        got[0, 3:6] = 0x7F
    np.testing.assert_array_equal(got, c[0, :, 0])
    np.testing.assert_array_equal(cache[2].cpu().numpy()[0, 0, :2], e[0, :, 0])


def test_rows_that_do_not_fit_are_not_written():
    B, T, Hkv, d, L_max = 4, 20, 2, 64, 32
    x = bf(normal_bf16(6, "k", (B, T, Hkv, d)))
    for start, rows, bit in (((13, 0, 0, 0), None, orth.DEVERR_CACHE_FULL), ((-1, 0, 0, 0), None, orth.DEVERR_POSITION),
                             ((0, 0, 0, 0), (21, 3, 3, 3), orth.DEVERR_POSITION),
                             ((0, 0, 0, 0), (-1, 3, 3, 3), orth.DEVERR_POSITION),
                             ((2147483647, 0, 0, 0), None, orth.DEVERR_CACHE_FULL)):
        cache = orth.kv_cache_q8(B, L_max, Hkv, d, dev())
        err = error_word()
        st, nr = (None if y is None else i32(np.array(y)) for y in (start, rows))
        orth.kv_quantize(x, x, *cache, start=st, rows=nr, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bit
        assert not raw(cache[0])[0].any() and raw(cache[0])[1:].any()


def test_strided_batches():
    """k, v as views of a longer buffer (a batch stride above dense), written and read back in place."""
    B, T, Hkv, d = 3, 37, 2, 128
    full = bf(normal_bf16(8, "k", (B, T + 11, Hkv, d)))
    view = full[:, :T]
    cache = orth.kv_cache_q8(B, T, Hkv, d, dev())
    orth.kv_quantize(view, view, *cache)
    dense = orth.kv_cache_q8(B, T, Hkv, d, dev())
    orth.kv_quantize(view.contiguous(), view.contiguous(), *dense)
    out = torch.zeros_like(full)
    orth.kv_dequantize(*cache, out[:, :T], torch.zeros_like(full)[:, :T])
    torch.cuda.synchronize()
    for a, b in zip(cache, dense):
        np.testing.assert_array_equal(raw(a), raw(b))
    assert not out[:, T:].any() and out[:, :T].any()


# ------------------------------------------------------------------------------ decode


class Q8Decode:
    """Device and oracle state of a batch whose caches hold codes."""

    def __init__(self, lens, steps, Hq, Hkv, d, window, code, seed):
        B = len(lens)
        L_max = (max(lens) + steps + 15) // 16 * 16
        cfg = DecodeConfig("q8", B=B, T0=max(max(lens), 1), steps=steps, Hq=Hq, Hkv=Hkv, d=d, window=window)
        self.cfg, self.inp, self.code, self.L_max = cfg, make_decode(cfg, seed), code, L_max
        self.codes = [np.full((B, L_max, Hkv, d), NAN_CODE, np.uint8) for _ in range(2)]
        self.exps = [np.full((B, L_max, Hkv), ANY_EXP, np.int8) for _ in range(2)]
        self.vals = [np.full((B, L_max, Hkv, d), 0x7FC0, np.uint16) for _ in range(2)]
        for i, src in enumerate((self.inp.k_cache, self.inp.v_cache)):
            for b, n in enumerate(lens):
                c, e = quantize(src[b, :n], code) if n else (None, None)
                if n:
                    self.codes[i][b, :n], self.exps[i][b, :n] = c, e
                    self.vals[i][b, :n] = value_bits(c, e, code)
        self.lens = np.array(lens, np.int32)
        self.dev_cache = [codes(c, code) for c in self.codes] + [exps(e) for e in self.exps]
        self.cl = i32(self.lens)
        self.vec = [f32(x) for x in (self.inp.alpha, self.inp.beta, self.inp.alpha_c, self.inp.beta_c)]
        self.ws = orth._binding.decode_q8_workspace(B, L_max, Hq, Hkv, d, dev())
        self.err = error_word()

    def step(self, i):
        n = self.inp
        return orth.decode_step_q8(bf(n.q_new[i]), bf(n.qc_new[i]), bf(n.k_new[i]), bf(n.v_new[i]), *self.dev_cache,
                                   self.cl, *self.vec, window=self.cfg.window, scale=self.cfg.scale,
                                   workspace=self.ws, dev_err=self.err)

    def oracle_step(self, i):
        n, new = self.inp, []
        for j, src in enumerate((n.k_new[i], n.v_new[i])):
            c, e = quantize(src, self.code)
            for b in range(len(self.lens)):
                self.codes[j][b, self.lens[b]], self.exps[j][b, self.lens[b]] = c[b], e[b]
            new.append(value_bits(c, e, self.code))
        return oracle.decode_step(n.q_new[i], n.qc_new[i], *new, *self.vals, self.lens, n.alpha, n.beta, n.alpha_c,
                                  n.beta_c, self.cfg.window, self.cfg.scale)

    def check_cache(self):
        for got, want in zip(self.dev_cache[:2], self.codes):
            np.testing.assert_array_equal(raw(got), want)
        for got, want in zip(self.dev_cache[2:], self.exps):
            np.testing.assert_array_equal(got.cpu().numpy(), want.transpose(0, 2, 1))
        np.testing.assert_array_equal(self.cl.cpu().numpy(), self.lens)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,steps,Hq,Hkv,d,window", [
    ((0,), 2, 2, 1, 64, 128),                               # an empty cache
    ((1,), 2, 4, 4, 128, 1),                                # G = 1, a window of the token itself
    ((62, 63, 64, 65), 3, 8, 2, 64, 64),                    # across a block's border, window of one block
    ((0, 1, 15, 16, 127, 128, 129, 1000, 4097), 2, 32, 8, 128, 128),
    ((300, 7), 2, 8, 4, 128, 300),                          # G = 2, a window longer than a cache
    ((517, 64), 2, 16, 2, 128, 77),                         # G = 8
    ((1200, 3), 2, 16, 1, 128, 5000),                       # G = 16, a window over everything
    ((700,), 2, 16, 1, 64, 129),
    ((9000,), 1, 32, 8, 128, 128),
])
def test_decode_steps_match_oracle(code, lens, steps, Hq, Hkv, d, window):
    s = Q8Decode(lens, steps, Hq, Hkv, d, window, code, 900 + len(lens) + d)
    for i in range(steps):
        o, oc = s.step(i)
        ro, roc = s.oracle_step(i)
        assert_parity(val(o), ro, f"step {i} base")
        assert_parity(val(oc), roc, f"step {i} copy")
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0
    s.check_cache()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_decode_with_rows_of_very_different_size(code):
    """Rows whose exponents span a wide range: values 2^-40 .. 2^40 in V, keys 2^-30 .. 2^4."""
    lens, Hq, Hkv, d = (400,), 8, 2, 64
    s = Q8Decode(lens, 1, Hq, Hkv, d, 128, code, 31)
    rng = np.random.default_rng(4)
    for i, (lo, hi) in enumerate(((-30, 3), (-40, 1))):
        s.exps[i][0, :400] = np.clip(s.exps[i][0, :400] + rng.integers(lo, hi, (400, Hkv)), -126, 127)
        s.vals[i][0, :400] = value_bits(s.codes[i][0, :400], s.exps[i][0, :400], code)
    s.dev_cache = [codes(c, code) for c in s.codes] + [exps(e) for e in s.exps]
    o, oc = s.step(0)
    ro, roc = s.oracle_step(0)
    assert_parity(val(o), ro, "base")
    assert_parity(val(oc), roc, "copy")
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 2), (2, 2)])
def test_decode_window_does_not_meet_what_lies_before_it(Hq, Hkv):
    """Rows before the base token's window hold NaN codes, up to the row next to it: the base output is the same."""
    out = []
    for nan in (False, True):
        s = Q8Decode((500, 150), 1, Hq, Hkv, 64, 100, "e4m3", 17)
        if nan:
            for b, n in enumerate((500, 150)):
                s.dev_cache[0].view(torch.int8)[b, :n - 99] = NAN_CODE
                s.dev_cache[1].view(torch.int8)[b, :n - 99] = NAN_CODE
        out.append(s.step(0))
    np.testing.assert_array_equal(bits(out[0][0]), bits(out[1][0]))
    assert torch.isfinite(out[0][1]).all() and torch.isnan(out[1][1]).all()


def test_decode_full_cache_writes_nothing():
    s = Q8Decode((14, 31), 3, 8, 2, 64, 128, "e4m3", 12)  # L_max = 48
    s.cl.copy_(i32(np.array([14, 48])))
    before = [raw(t).copy() for t in s.dev_cache]
    o, oc = s.step(0)
    torch.cuda.synchronize()
    assert int(s.err.item()) == orth.DEVERR_CACHE_FULL
    np.testing.assert_array_equal(s.cl.cpu().numpy(), [15, 48])
    assert not o[1].any() and not oc[1].any() and o[0].any() and oc[0].any()
    after = [raw(t) for t in s.dev_cache]
    for x, y in zip(before, after):
        np.testing.assert_array_equal(x[1], y[1])
    s.cl.copy_(i32(np.array([-1, 15])))  # a length below zero likewise, the other sequence runs on
    o, oc = s.step(1)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(s.cl.cpu().numpy(), [-1, 16])
    assert not o[0].any() and not oc[0].any() and o[1].any()


@pytest.mark.parametrize("shift", [24, -24])
def test_decode_with_large_and_small_queries(shift):
    """Queries 2^24 times larger (or smaller) against keys as much smaller (larger): the same logits as without."""
    s = Q8Decode((200,), 1, 8, 2, 64, 128, "e4m3", 13)
    s.exps[0][0, :200] -= shift
    s.vals[0][0, :200] = value_bits(s.codes[0][0, :200], s.exps[0][0, :200], "e4m3")
    s.inp.k_new[0] = value_bits(*(lambda c, e: (c, e - shift))(*quantize(s.inp.k_new[0], "e4m3")), "e4m3")
    for n in ("alpha", "beta", "alpha_c", "beta_c"):
        getattr(s.inp, n)[...] *= np.float32(2.0 ** shift)
    s.vec = [f32(x) for x in (s.inp.alpha, s.inp.beta, s.inp.alpha_c, s.inp.beta_c)]
    s.dev_cache = [codes(c, "e4m3") for c in s.codes] + [exps(e) for e in s.exps]
    o, oc = s.step(0)
    ro, roc = s.oracle_step(0)
    assert_parity(val(o), ro, "base")
    assert_parity(val(oc), roc, "copy")
    assert int(s.err.item()) == 0


def test_decode_is_repeatable_on_other_streams_and_in_graphs():
    """The same step gives the same bits: eagerly, on another stream, and replayed from a captured graph; two
    batches with workspaces of their own run at once."""
    def fresh():
        return Q8Decode((777, 64, 0), 1, 32, 8, 128, 128, "e4m3", 14)
    a, b, c = fresh(), fresh(), fresh()
    o1, oc1 = a.step(0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        o2, oc2 = b.step(0)
    with torch.cuda.stream(s2):
        o3, oc3 = c.step(0)
    torch.cuda.synchronize()
    for x, y in ((o1, o2), (o1, o3), (oc1, oc2), (oc1, oc3)):
        np.testing.assert_array_equal(bits(x), bits(y))
    # a captured step: every replay appends the next row; the lengths are put back in between
    g = fresh()
    n = g.inp
    args = [bf(n.q_new[0]), bf(n.qc_new[0]), bf(n.k_new[0]), bf(n.v_new[0])]
    out = [torch.empty_like(o1), torch.empty_like(oc1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orth.decode_step_q8(*args, *g.dev_cache, g.cl, *g.vec, window=128, scale=g.cfg.scale, o=out[0], oc=out[1],
                            workspace=g.ws, dev_err=g.err)
    for _ in range(3):
        g.cl.copy_(i32(np.array([777, 64, 0])))
        out[0].zero_(), out[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(out[0]), bits(o1))
        np.testing.assert_array_equal(bits(out[1]), bits(oc1))
        np.testing.assert_array_equal(g.cl.cpu().numpy(), [778, 65, 1])


def test_decode_offsets_beyond_32_bits():
    """Sequences whose rows lie more than 2^31 (and 2^32) codes into the cache's buffer."""
    B, L_max, Hq, Hkv, d, n = 5, 1 << 20, 8, 8, 128, 300
    s = Q8Decode((n,) * B, 1, Hq, Hkv, d, 128, "e4m3", 15)
    big = orth.kv_cache_q8(B, L_max, Hkv, d, dev())
    for t, src in zip(big[:2], s.dev_cache[:2]):
        t.view(torch.int8)[:, :n].copy_(src.view(torch.int8)[:, :n])
    for t, src in zip(big[2:], s.dev_cache[2:]):
        t[:, :, :n].copy_(src[:, :, :n])
    small = s.dev_cache
    s.dev_cache, s.ws = list(big), orth._binding.decode_q8_workspace(B, L_max, Hq, Hkv, d, dev())
    o, oc = s.step(0)
    ro, roc = s.oracle_step(0)
    assert_parity(val(o), ro, "base")
    assert_parity(val(oc), roc, "copy")
    k = torch.empty((B, 301, Hkv, d), dtype=torch.bfloat16, device=dev())
    v = torch.empty_like(k)
    orth.kv_dequantize(*big, k, v)
    np.testing.assert_array_equal(bits(k)[:, :301], s.vals[0][:, :301])
    np.testing.assert_array_equal(bits(v)[:, :301], s.vals[1][:, :301])
    # the last rows of the last sequence, written and read back
    x = normal_bf16(16, "k", (B, 8, Hkv, d))
    st = i32(np.full(B, L_max - 8))
    orth.kv_quantize(bf(x), bf(x), *big, start=st)
    back = torch.empty((B, 8, Hkv, d), dtype=torch.bfloat16, device=dev())
    orth.kv_dequantize(*big, back, torch.empty_like(back), start=st)
    np.testing.assert_array_equal(bits(back), value_bits(*quantize(x, "e4m3"), "e4m3"))
    del small


def test_prompt_then_decode_over_one_cache():
    """Used together: a prompt's K/V go into the cache chunk by chunk, tokens are decoded behind it, and the read
    back cache gives the framework's bf16 decode step the same answers."""
    B, T, Hq, Hkv, d, steps = 2, 150, 8, 2, 128, 3
    k, v = (normal_bf16(40, n, (B, T, Hkv, d)) for n in ("k", "v"))
    cache = orth.kv_cache_q8(B, T + steps, Hkv, d, dev())
    L_max = cache[0].shape[1]
    kd, vd = bf(k), bf(v)
    for a in range(0, T, 64):
        rows = kd[:, a:a + 64]
        orth.kv_quantize(rows, vd[:, a:a + 64], *cache, start=i32(np.full(B, a)))
    kb = torch.zeros((B, L_max, Hkv, d), dtype=torch.bfloat16, device=dev())
    vb = torch.zeros_like(kb)
    orth.kv_dequantize(*cache, kb, vb, rows=i32(np.full(B, T)))
    inp = make_decode(DecodeConfig("x", B=B, T0=1, steps=steps, Hq=Hq, Hkv=Hkv, d=d), 41)
    vec = [f32(x) for x in (inp.alpha, inp.beta, inp.alpha_c, inp.beta_c)]
    cl, clb = i32(np.full(B, T)), i32(np.full(B, T))
    for i in range(steps):
        q, qc = bf(inp.q_new[i]), bf(inp.qc_new[i])
        o, oc = orth.decode_step_q8(q, qc, bf(inp.k_new[i]), bf(inp.v_new[i]), *cache, cl, *vec)
        new = [bf(value_bits(*quantize(x, "e4m3"), "e4m3")) for x in (inp.k_new[i], inp.v_new[i])]
        rk, rv = kb.clone(), vb.clone()
        ob, ocb = orth.decode_step(q, qc, *new, kb, vb, clb, *vec)
        ro, roc = oracle.decode_step(inp.q_new[i], inp.qc_new[i], bits(new[0]), bits(new[1]), bits(rk), bits(rv),
                                     np.full(B, T + i, np.int32), inp.alpha, inp.beta, inp.alpha_c, inp.beta_c, 128,
                                     1 / math.sqrt(d))
        for x, w in ((o, ro), (ob, ro), (oc, roc), (ocb, roc)):
            assert_parity(val(x), w, f"step {i}")
    check = torch.zeros_like(kb)
    orth.kv_dequantize(*cache, check, torch.zeros_like(kb), rows=i32(np.full(B, T + steps)))
    np.testing.assert_array_equal(bits(check), bits(kb))
