"""GPU tests of the attention behind a shared prompt prefix (copies and decode step) against the fp64 oracle, which
takes each sequence's prefix and own rows as one sequence."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
import oracle
from synthetic import DecodeConfig, make_decode, normal_bf16, scale_offset
from tests.gpu_util import assert_parity, bf, bits, dev, f32, i32, val

pytestmark = pytest.mark.gpu


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=dev())


class Copies:
    def __init__(self, B, T_out, P, T_kv, Hq, Hkv, d, seed):
        self.kp, self.vp = (normal_bf16(seed + 5000, n, (P, Hkv, d)) for n in ("k", "v"))
        self.k, self.v = (normal_bf16(seed, n, (B, T_kv, Hkv, d)) for n in ("k", "v"))
        self.qc = normal_bf16(seed, "qc_raw", (B, T_out, Hq, d))
        self.pos = np.random.default_rng(seed).integers(0, T_kv, (B, T_out)).astype(np.int32)
        self.pos[0, 0], self.pos[-1, -1] = T_kv - 1, 0
        self.ac, self.bc = scale_offset(seed, Hq, d, prefix="_c")
        self.scale, self.P = d ** -0.5, P

    def oracle(self):
        B = len(self.k)
        k, v = (np.concatenate([np.broadcast_to(p[None], (B,) + p.shape), x], 1)
                for p, x in ((self.kp, self.k), (self.vp, self.v)))
        return oracle.xattn(self.qc, self.pos + self.P, k, v, self.ac, self.bc, self.scale)

    def run(self, **kw):
        return orth.xattn_prefix_fwd(bf(self.qc), i32(self.pos), bf(self.kp), bf(self.vp), bf(self.k), bf(self.v),
                                     f32(self.ac), f32(self.bc), scale=self.scale, **kw)


@pytest.mark.parametrize("B,T_out,P,T_kv,Hq,Hkv,d", [
    (1, 1, 1, 1, 2, 1, 64),              # one row on each side
    (2, 1, 63, 65, 4, 4, 128),           # G = 1
    (3, 1, 129, 7, 8, 2, 64),            # a few rows, ragged prefix
    (8, 1, 2000, 130, 32, 8, 128),       # 32 rows a KV head
    (5, 3, 700, 64, 8, 4, 128),          # G = 2, rows of a tile from several sequences
    (2, 5, 1000, 500, 16, 1, 128),       # G = 16
    (33, 1, 513, 40, 8, 2, 128),         # 132 rows: a second, almost empty tile
    (64, 1, 1500, 20, 32, 8, 128),       # 256 rows
    (2, 70, 900, 333, 8, 2, 64),         # own part beyond 256 rows
    (3, 40, 300, 100, 16, 2, 128),       # G = 8
    (1, 300, 450, 310, 8, 2, 128),
    (1, 260, 100, 300, 2, 2, 64),        # G = 1, many copies
    (4, 1, 20000, 64, 8, 1, 128),        # a long prefix, one KV head
    (2, 320, 333, 400, 32, 8, 128),      # many copies a sequence: prefix and own rows in one pass
    (5, 60, 129, 61, 64, 8, 64),         # the same with G = 8, a padded tile
    (5, 400, 70, 500, 8, 8, 64),         # G = 1
    (7, 48, 1, 130, 64, 4, 128),         # G = 16
    (10, 250, 64, 64, 16, 8, 128),       # G = 2
])
def test_copies_match_oracle(B, T_out, P, T_kv, Hq, Hkv, d):
    c = Copies(B, T_out, P, T_kv, Hq, Hkv, d, 200 + P)
    err = error_word()
    got = c.run(dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert_parity(val(got), c.oracle(), "copies")


@pytest.mark.parametrize("B,T_out,Hq,Hkv", [(2, 3, 8, 2), (16, 1, 32, 8), (2, 80, 8, 2), (10, 62, 32, 8), (2, 1, 16, 1)])
def test_copies_out_of_range_are_zero_and_reported(B, T_out, Hq, Hkv):
    c = Copies(B, T_out, 300, 50, Hq, Hkv, 128, 21)
    ref = c.oracle()
    c.pos[0, 0], c.pos[-1, -1] = -1, 50
    err = error_word()
    got = val(c.run(dev_err=err))
    assert int(err.item()) == orth.DEVERR_POSITION
    assert not got[0, 0].any() and not got[-1, -1].any()
    ref[0, 0], ref[-1, -1] = 0, 0
    assert_parity(got, ref, "the others")


@pytest.mark.parametrize("B,T_out,Hq,Hkv,used", [(10, 64, 32, 8, 130), (10, 64, 32, 8, 64), (3, 1, 8, 2, 100),
                                                  (40, 1, 8, 1, 65), (1, 1, 2, 2, 1), (2, 2, 8, 2, 101),
                                                  (3, 3, 8, 2, 70), (2, 5, 16, 1, 290), (1, 30, 8, 2, 17)])
def test_rows_behind_the_last_position_do_not_matter(B, T_out, Hq, Hkv, used):
    """Own rows that no copy of the batch has reached hold NaN."""
    c = Copies(B, T_out, 200, 300, Hq, Hkv, 128, 24)
    c.pos = np.minimum(c.pos, used - 1)
    c.pos[:, 0] = used - 1
    k, v = c.k.copy(), c.v.copy()
    k[:, used:], v[:, used:] = 0x7FC0, 0x7FC0
    got = orth.xattn_prefix_fwd(bf(c.qc), i32(c.pos), bf(c.kp), bf(c.vp), bf(k), bf(v), f32(c.ac), f32(c.bc), scale=c.scale)
    assert_parity(val(got), c.oracle(), "copies")


@pytest.mark.parametrize("B,T_out,P,Hq,Hkv", [(2, 1, 300, 8, 2), (3, 3, 300, 8, 2), (2, 2, 20000, 8, 2), (3, 3, 20000, 8, 2),
                                              (40, 1, 300, 8, 2), (4, 1, 3000, 16, 1), (2, 80, 300, 8, 2), (10, 62, 300, 32, 8)])
@pytest.mark.parametrize("where", ["prefix key", "prefix value", "own key", "own value", "query"])
def test_nan_reaches_the_rows_that_see_it_and_no_other(where, B, T_out, P, Hq, Hkv):
    """A NaN value row is 0 * NaN for the copies of its sequence that lie before it: those may be NaN too."""
    c = Copies(B, T_out, P, 200, Hq, Hkv, 128, 25)
    c.pos[-1, 0] = 150
    ref = c.oracle()
    sees = np.zeros((B, T_out, Hq), bool)
    any_of = np.zeros((B, T_out, Hq), bool)
    if where == "query":
        c.qc[0, 0, 1, 7] = 0x7FC0
        sees[0, 0, 1] = True
    elif where.startswith("prefix"):
        (c.kp if where == "prefix key" else c.vp)[150, 0, :] = 0x7FC0
        sees[:, :, :Hq // Hkv] = True
    else:
        (c.k if where == "own key" else c.v)[-1, 5, 0, :] = 0x7FC0
        sees[-1, c.pos[-1] >= 5, :Hq // Hkv] = True
        any_of[-1, :, :Hq // Hkv] = where == "own value"
    got = val(c.run())
    assert np.isnan(got[sees]).all()
    others = ~(sees | any_of)
    assert_parity(got[others], ref[others], "the others")


@pytest.mark.parametrize("B,T_out,Hq,Hkv", [(3, 2, 8, 2), (5, 1, 8, 2), (10, 64, 32, 8)])
def test_copies_strided_and_repeatable(B, T_out, Hq, Hkv):
    """Batch strides above dense for queries, own rows and output; the bits do not depend on strides, stream or
    what the workspace held."""
    P, T_kv, d = 800, 70, 128
    c = Copies(B, T_out, P, T_kv, Hq, Hkv, d, 22)
    ref = bits(c.run())

    def wide(x, n):
        y = torch.full((B, x.shape[1] + n) + x.shape[2:], float("nan"), dtype=torch.bfloat16, device=dev())
        y[:, :x.shape[1]] = bf(x)
        return y[:, :x.shape[1]]
    out = torch.full((B, T_out + 1, Hq, d), 3.0, dtype=torch.bfloat16, device=dev())
    n = orth.xattn_prefix_workspace_size(B, T_out, P, T_kv, Hq, Hkv, d)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (wide(c.qc, 3), i32(c.pos), bf(c.kp), bf(c.vp), wide(c.k, 5), wide(c.v, 5), f32(c.ac), f32(c.bc))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        orth.xattn_prefix_fwd(*args, scale=c.scale, out=out[:, :T_out], workspace=ws)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(out[:, :T_out]), ref)
    assert (out[:, T_out:] == 3.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orth.xattn_prefix_fwd(*args, scale=c.scale, out=out[:, :T_out], workspace=ws)
    for _ in range(2):
        out.zero_(), ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(out[:, :T_out]), ref)


@pytest.mark.parametrize("rows", [1, 16, 40, 300, -1])
def test_copies_with_large_keys(rows):
    """Keys four times as large at a few rows (logits that decide) and key rows beyond fp16's range against small
    queries, in the prefix and among the own rows."""
    B, P, T_kv, Hq, Hkv, d = rows, 500, 66, 4, 1, 128
    T_out = 1
    if rows < 0:  # many copies a sequence
        B, T_out, Hq, Hkv = 10, 64, 32, 8
    c = Copies(B, T_out, P, T_kv, Hq, Hkv, d, 23)
    c.kp[100], c.k[:, 3] = c.kp[100] + (2 << 7), c.k[:, 3] + (2 << 7)  # exponent + 2
    c.kp[200, :, 5] = 0x4800  # 2^17 in one column
    c.k[:, 10, :, 5] = 0x4800
    c.qc[..., 5] = 0x3600     # 2^-19
    c.bc[:, 5] = 0
    got = c.run()
    assert_parity(val(got), c.oracle(), "large keys")


class PrefixDecode:
    def __init__(self, lens, steps, P, Hq, Hkv, d, window, seed, spare=0):
        B = len(lens)
        self.cfg = DecodeConfig("p", B=B, T0=max(max(lens), 1), steps=steps, Hq=Hq, Hkv=Hkv, d=d, window=window)
        self.inp = make_decode(self.cfg, seed)
        self.P, L_max = P, max(lens) + steps + spare
        self.kp, self.vp = (normal_bf16(seed + 5000, n, (P, Hkv, d)) for n in ("k", "v"))
        self.k, self.v = (np.full((B, P + L_max, Hkv, d), 0x7FC0, np.uint16) for _ in range(2))
        for x, p, src in ((self.k, self.kp, self.inp.k_cache), (self.v, self.vp, self.inp.v_cache)):
            x[:, :P] = p
            for b, n in enumerate(lens):
                x[b, P:P + n] = src[b, :n]
        self.lens = np.array(lens, np.int32)
        self.total = self.lens + np.int32(P)
        self.cl = i32(self.lens)
        self.dk, self.dv = bf(self.k[:, P:]), bf(self.v[:, P:])
        self.dkp, self.dvp = bf(self.kp), bf(self.vp)
        self.vec = [f32(x) for x in (self.inp.alpha, self.inp.beta, self.inp.alpha_c, self.inp.beta_c)]
        self.ws = orth._binding.decode_prefix_workspace(B, P, L_max, Hq, Hkv, d, dev())
        self.err = error_word()

    def step(self, i, **kw):
        n = self.inp
        return orth.decode_step_prefix(bf(n.q_new[i]), bf(n.qc_new[i]), bf(n.k_new[i]), bf(n.v_new[i]), self.dkp,
                                       self.dvp, self.dk, self.dv, self.cl, *self.vec, window=self.cfg.window,
                                       scale=self.cfg.scale, workspace=self.ws, dev_err=self.err, **kw)

    def oracle_step(self, i):
        n = self.inp
        return oracle.decode_step(n.q_new[i], n.qc_new[i], n.k_new[i], n.v_new[i], self.k, self.v, self.total, n.alpha,
                                  n.beta, n.alpha_c, n.beta_c, self.cfg.window, self.cfg.scale)


@pytest.mark.parametrize("lens,steps,P,Hq,Hkv,d,window", [
    ((0,), 2, 1, 2, 1, 64, 128),                       # one prefix row, nothing of its own
    ((0, 1, 5), 3, 127, 4, 4, 128, 128),               # the window reaches into the prefix
    ((63, 64, 65, 126, 127, 128), 2, 64, 8, 2, 64, 128),
    ((10, 300, 0, 77), 2, 1000, 32, 8, 128, 300),
    ((3,) * 8, 2, 5000, 32, 8, 128, 128),              # 32 rows a KV head
    ((2, 40, 130), 2, 333, 16, 1, 128, 5000),          # G = 16, a window over everything
    ((5, 6), 2, 190, 16, 2, 64, 1),                    # G = 8
    (tuple(range(64)), 1, 700, 32, 8, 128, 128),       # 256 rows
    (tuple(range(0, 330, 10)), 1, 1025, 8, 4, 128, 64),  # G = 2, 66 rows
    ((20,), 2, 30000, 8, 1, 128, 128),
])
def test_decode_steps_match_oracle(lens, steps, P, Hq, Hkv, d, window):
    s = PrefixDecode(lens, steps, P, Hq, Hkv, d, window, 400 + P)
    for i in range(steps):
        o, oc = s.step(i)
        ro, roc = s.oracle_step(i)
        assert_parity(val(o), ro, f"step {i} base")
        assert_parity(val(oc), roc, f"step {i} copy")
    assert int(s.err.item()) == 0
    np.testing.assert_array_equal(bits(s.dk), s.k[:, P:])
    np.testing.assert_array_equal(bits(s.dv), s.v[:, P:])
    np.testing.assert_array_equal(bits(s.dkp), s.kp)
    np.testing.assert_array_equal(s.cl.cpu().numpy() + P, s.total)


def test_one_workspace_serves_batches_of_other_sizes():
    """A workspace of the largest batch goes from step to step of other batches, and through two captured graphs
    that run in turn; the bits are those of a workspace of one's own."""
    shapes = [((700, 3, 64, 900), 500, 8, 2, 128), ((40,), 9000, 16, 1, 128), ((5, 1300), 70, 4, 4, 64)]
    make = [lambda s=s, i=i: PrefixDecode(s[0], 1, s[1], s[2], s[3], s[4], 128, 60 + i) for i, s in enumerate(shapes)]
    want = [[bits(x) for x in m().step(0)] for m in make]
    big = max((m().ws.nbytes for m in make))
    ws = torch.zeros(big, dtype=torch.uint8, device=dev())
    runs = [m() for m in make]
    for r in runs:
        r.ws = ws
    for i in (0, 2, 1, 0, 1, 2):
        runs[i].cl.copy_(i32(runs[i].lens))
        for got, ref in zip(runs[i].step(0), want[i]):
            np.testing.assert_array_equal(bits(got), ref)
    graphs, outs = [], []
    for r in runs:
        r.cl.copy_(i32(r.lens))
        new = [bf(x) for x in (r.inp.q_new[0], r.inp.qc_new[0], r.inp.k_new[0], r.inp.v_new[0])]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = orth.decode_step_prefix(*new, r.dkp, r.dvp, r.dk, r.dv, r.cl, *r.vec, window=r.cfg.window,
                                        scale=r.cfg.scale, workspace=ws, dev_err=r.err)
        graphs.append((g, new)), outs.append(o)
    for i in (1, 0, 2, 0, 1):
        runs[i].cl.copy_(i32(runs[i].lens))
        graphs[i][0].replay()
        for got, ref in zip(outs[i], want[i]):
            np.testing.assert_array_equal(bits(got), ref)
    assert all(int(r.err.item()) == 0 for r in runs)


def test_wrong_error_words_and_workspaces_are_refused():
    s = PrefixDecode((3, 4), 1, 100, 8, 2, 64, 128, 61)
    for bad in (torch.zeros(1, dtype=torch.uint8, device=dev()), torch.zeros(0, dtype=torch.int32, device=dev()),
                torch.zeros(1, dtype=torch.int32)):
        s.err = bad
        with pytest.raises(orth.OrthrosError):
            s.step(0)
    s.err = None
    for bad in (s.ws[:-256], s.ws.cpu(), s.ws[16:]):
        s.ws = bad
        with pytest.raises(orth.OrthrosError):
            s.step(0)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 2)])
@pytest.mark.parametrize("lens,P,window", [((200, 77), 300, 100), ((20, 64), 130, 90)])
def test_decode_window_does_not_meet_what_lies_before_it(Hq, Hkv, lens, P, window):
    """Rows before the base token's window hold NaN, up to the row next to it: the base output does not change."""
    s = PrefixDecode(lens, 1, P, Hq, Hkv, 128, window, 16)
    o, _ = s.step(0)
    t = PrefixDecode(lens, 1, P, Hq, Hkv, 128, window, 16)
    first = [P + n - window + 1 for n in lens]  # the window's first row, counted through prefix and own rows
    for b, f in enumerate(first):
        t.dk[b, :max(0, f - P)] = float("nan")
        t.dv[b, :max(0, f - P)] = float("nan")
    t.dkp[:min(first)] = float("nan")
    t.dvp[:min(first)] = float("nan")
    o2, oc2 = t.step(0)
    np.testing.assert_array_equal(bits(o), bits(o2))
    assert torch.isnan(oc2).all()
    ro, _ = s.oracle_step(0)
    assert_parity(val(o2), ro, "base")


@pytest.mark.parametrize("B", [2, 40])
def test_decode_full_cache_writes_nothing(B):
    s = PrefixDecode((14,) * B, 1, 100, 8, 2, 64, 128, 12)
    s.cl.copy_(i32(np.array([15] + [14] * (B - 2) + [-3])))
    before = bits(s.dk)
    o, oc = s.step(0)
    torch.cuda.synchronize()
    assert int(s.err.item()) == orth.DEVERR_CACHE_FULL
    np.testing.assert_array_equal(s.cl.cpu().numpy(), [15] + [15] * (B - 2) + [-3])
    for b in (0, B - 1):
        assert not o[b].any() and not oc[b].any()
        np.testing.assert_array_equal(bits(s.dk)[b], before[b])


def test_decode_is_repeatable_on_other_streams_and_in_graphs():
    def fresh():
        return PrefixDecode((700, 64, 0, 9, 33), 1, 3000, 32, 8, 128, 128, 14)
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
    g = fresh()
    n = g.inp
    args = [bf(n.q_new[0]), bf(n.qc_new[0]), bf(n.k_new[0]), bf(n.v_new[0])]
    out = [torch.empty_like(o1), torch.empty_like(oc1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orth.decode_step_prefix(*args, g.dkp, g.dvp, g.dk, g.dv, g.cl, *g.vec, window=128, scale=g.cfg.scale, o=out[0],
                                oc=out[1], workspace=g.ws, dev_err=g.err)
    for _ in range(3):
        g.cl.copy_(i32(g.lens))
        out[0].zero_(), out[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(out[0]), bits(o1))
        np.testing.assert_array_equal(bits(out[1]), bits(oc1))
        np.testing.assert_array_equal(g.cl.cpu().numpy(), g.lens + 1)
    # many steps behind one another without a wait, against the oracle at the end
    s = PrefixDecode((5, 60, 0), 12, 200, 8, 2, 128, 128, 15)
    outs = [s.step(i) for i in range(12)]
    for i in range(12):
        ro, roc = s.oracle_step(i)
        assert_parity(val(outs[i][0]), ro, f"step {i} base")
        assert_parity(val(outs[i][1]), roc, f"step {i} copy")


def test_prompts_behind_a_prefix_then_decode():
    """Used together: the last prompt position of every sequence attends by xattn_prefix_fwd, then tokens are decoded
    behind the same prefix and own rows; the copy's answer at position p is the same operator's either way."""
    B, P, T, Hq, Hkv, d = 4, 300, 40, 8, 2, 128
    c = Copies(B, 1, P, T, Hq, Hkv, d, 50)
    c.pos[:] = T - 1
    whole = c.run()
    inp = make_decode(DecodeConfig("x", B=B, T0=1, steps=1, Hq=Hq, Hkv=Hkv, d=d), 51)
    k, v = (torch.cat([x[:, :T - 1], torch.zeros_like(x[:, :3])], 1) for x in (bf(c.k), bf(c.v)))
    cl = i32(np.full(B, T - 1))
    ones, zeros = f32(np.ones((Hq, d), np.float32)), f32(np.zeros((Hq, d), np.float32))
    o, oc = orth.decode_step_prefix(bf(inp.q_new[0]), bf(c.qc[:, 0]), bf(c.k[:, T - 1]), bf(c.v[:, T - 1]), bf(c.kp),
                                    bf(c.vp), k, v, cl, ones, zeros, f32(c.ac), f32(c.bc), scale=c.scale)
    ref = c.oracle()
    assert_parity(val(whole), ref, "prompt")
    assert_parity(val(oc), ref[:, 0], "decode")
    np.testing.assert_array_equal(bits(k)[:, :T], c.k)
