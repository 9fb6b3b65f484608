"""GPU tests of drafted trees over a cache, and of what is accepted of them, against plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
import oracle
from synthetic import bf16_to_f32, normal_bf16, scale_offset
from tests import sink_util
from tests.attend_util import assert_bounded
from tests.gpu_util import assert_parity, bf, bits, dev, f32, i32, val

pytestmark = pytest.mark.gpu
NAN = 0x7FC0


def f64(x):
    return bf16_to_f32(x).astype(np.float64)


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=dev())


def parents(rng, B, N, shape):
    if shape == "chain":
        return np.tile(np.arange(-1, N - 1), (B, 1)).astype(np.int32)
    if shape == "star":
        return np.full((B, N), -1, np.int32)
    return np.stack([[rng.integers(-1, i) if i else -1 for i in range(N)] for _ in range(B)]).astype(np.int32)


class Tree:
    def __init__(self, B, N, L, Hq, Hkv, d, window=128, sinks=0, shape="random", ragged=False, seed=1, room=0):
        rng = np.random.default_rng(seed)
        self.x, self.xc = (normal_bf16(seed, n, (B, N, Hq, d)) for n in ("q_raw", "qc_raw"))
        self.kn, self.vn = (normal_bf16(seed + 1000, n, (B, N, Hkv, d)) for n in ("k", "v"))
        self.L_max = max(1, L + room)
        self.k, self.v = (normal_bf16(seed, n, (B, self.L_max, Hkv, d)) for n in ("k", "v"))
        self.vec = (*scale_offset(seed, Hq, d), *scale_offset(seed, Hq, d, prefix="_c"))
        self.parent = parents(rng, B, N, shape)
        self.lens = np.full(B, L, np.int32)
        self.nodes = None
        if ragged:
            self.lens = rng.integers(0, L + 1, B).astype(np.int32)
            self.nodes = rng.integers(0, N + 1, B).astype(np.int32)
            self.lens[0], self.nodes[0] = L, N
        self.window, self.sinks = window, sinks

    def reference(self):
        return sink_util.tree(f64(self.x), f64(self.xc), f64(self.kn), f64(self.vn), self.parent, f64(self.k), f64(self.v),
                              self.lens, [a.astype(np.float64) for a in self.vec], self.window, self.sinks, self.nodes)

    def args(self):
        return (bf(self.x), bf(self.xc), bf(self.kn), bf(self.vn), i32(self.parent), bf(self.k), bf(self.v), i32(self.lens),
                *[f32(a) for a in self.vec])

    def run(self, **kw):
        return orth.decode_tree(*self.args(), window=self.window, sinks=self.sinks,
                                nodes=None if self.nodes is None else i32(self.nodes), **kw)

    def check(self, got):
        B, N = self.parent.shape
        for y, (ref, bound), what in zip(got, self.reference(), ("o", "oc")):
            y = val(y)
            for b in range(B):
                n = N if self.nodes is None else self.nodes[b]
                if n:
                    assert_bounded(y[b, :n], ref[b, :n], bound[b, :n] + 1e-30, f"{what}, sequence {b}")


@pytest.mark.parametrize("B,N,L,Hq,Hkv,d,window,sinks,shape,ragged", [
    (1, 1, 0, 2, 1, 64, 128, 0, "chain", False),       # nothing cached, one node
    (1, 1, 1, 2, 1, 64, 1, 1, "chain", False),
    (1, 1, 300, 4, 4, 128, 128, 4, "chain", False),    # G = 1: the single token of a layer with sinks
    (2, 1, 5000, 32, 8, 128, 128, 4, "chain", False),
    (1, 5, 300, 8, 2, 64, 128, 0, "chain", False),
    (2, 4, 129, 4, 2, 128, 2, 3, "chain", False),      # the window ends inside the tree
    (3, 8, 64, 2, 2, 128, 3, 30, "random", False),
    (2, 8, 10, 2, 2, 64, 4, 14, "chain", False),       # sinks that lie in the tree
    (1, 16, 777, 16, 1, 128, 128, 0, "random", False),  # 256 rows a KV head
    (2, 16, 1000, 32, 8, 128, 128, 0, "random", False),
    (4, 64, 500, 32, 8, 128, 128, 4, "random", True),
    (2, 64, 200, 16, 1, 64, 40, 16, "random", True),    # 1024 rows a KV head
    (3, 64, 130, 4, 4, 64, 10, 2, "chain", True),       # a chain that outgrows the window
    (2, 63, 300, 8, 1, 128, 300, 0, "star", True),
    (9, 7, 900, 8, 2, 128, 77, 5, "random", True),
    (33, 3, 70, 8, 4, 128, 33, 1, "random", True),      # more sequences than a warp's lanes
    (70, 2, 40, 2, 1, 64, 16, 0, "random", True),
    (1, 33, 20000, 4, 1, 128, 128, 4, "random", False),  # a long cache of one KV head
    (1, 3, 20000, 2, 1, 128, 1000, 4, "random", False),
    (2, 20, 0, 8, 2, 128, 128, 4, "random", False),
])
def test_tree_matches(B, N, L, Hq, Hkv, d, window, sinks, shape, ragged):
    c = Tree(B, N, L, Hq, Hkv, d, window, sinks, shape, ragged, seed=N + L, room=N)
    err = error_word()
    c.check(c.run(dev_err=err))
    assert int(err.item()) == 0


@pytest.mark.parametrize("N,Hq,Hkv", [(3, 8, 2), (9, 8, 2), (40, 8, 2), (64, 16, 2)])
@pytest.mark.parametrize("sinks", [0, 4])
def test_what_no_node_sees_may_hold_anything(N, Hq, Hkv, sinks):
    """NaN in cache rows behind the last, in K and V and queries of nodes behind a tree's last, and their parents;
    output rows there stay as they are."""
    B, L, d = 3, 500, 128
    c = Tree(B, N, L, Hq, Hkv, d, 60, sinks, ragged=True, seed=21, room=70)
    ref = c.run()
    o0, oc0 = (torch.full((B, N, Hq, d), 5.0, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    k, v, kn, vn, x, xc, parent = c.k.copy(), c.v.copy(), c.kn.copy(), c.vn.copy(), c.x.copy(), c.xc.copy(), c.parent.copy()
    for b in range(B):
        n = c.nodes[b]
        k[b, c.lens[b]:], v[b, c.lens[b]:] = NAN, NAN
        kn[b, n:], vn[b, n:], x[b, n:], xc[b, n:], parent[b, n:] = NAN, NAN, NAN, NAN, 99
    c2 = Tree(B, N, L, Hq, Hkv, d, 60, sinks, ragged=True, seed=21, room=70)
    c2.k, c2.v, c2.kn, c2.vn, c2.x, c2.xc, c2.parent = k, v, kn, vn, x, xc, parent
    err = error_word()
    got = c2.run(o=o0, oc=oc0, dev_err=err)
    assert int(err.item()) == 0
    for y, r in zip(got, ref):
        for b in range(B):
            n = c.nodes[b]
            np.testing.assert_array_equal(bits(y[b, :n]), bits(r[b, :n]))
            assert (y[b, n:] == 5.0).all()


@pytest.mark.parametrize("N,Hq,Hkv", [(3, 8, 2), (33, 8, 2)])
def test_rows_before_the_window_do_not_reach_the_base_tokens(N, Hq, Hkv):
    c = Tree(1, N, 700, Hq, Hkv, 128, 100, 4, seed=22)
    ref = c.run()[0]
    c.v[:, 4:600] = NAN
    c.k[:, 4:600] = NAN
    np.testing.assert_array_equal(bits(c.run()[0]), bits(ref))


@pytest.mark.parametrize("N,Hq,Hkv", [(6, 8, 2), (40, 8, 2)])
def test_bad_parents_nodes_and_lengths(N, Hq, Hkv):
    """Zeros for them and what hangs below them, an error bit, and the others as ever."""
    c = Tree(3, N, 200, Hq, Hkv, 64, seed=23)
    c.parent[0, 2], c.parent[0, 4], c.parent[1, 3] = 2, 2, -2
    err = error_word()
    got = c.run(dev_err=err)
    assert int(err.item()) == orth.DEVERR_POSITION
    c.check(got)
    assert not val(got[1])[0, 2].any() and not val(got[0])[0, 4].any() and not val(got[1])[1, 3].any()
    c = Tree(3, N, 200, Hq, Hkv, 64, seed=23)
    c.nodes = np.array([N, N + 1, -1], np.int32)
    err = error_word()
    got = [val(y) for y in c.run(dev_err=err)]
    assert int(err.item()) == orth.DEVERR_POSITION
    assert got[0][0].any() and not got[0][1:].any() and not got[1][1:].any()
    c.nodes = None
    c.lens[1:] = [-1, 201]
    err = error_word()
    got = [val(y) for y in c.run(dev_err=err)]
    assert int(err.item()) == orth.DEVERR_CACHE_FULL
    assert got[0][0].any() and not got[0][1:].any() and not got[1][1:].any()


@pytest.mark.parametrize("N,Hq,Hkv", [(2, 8, 2), (5, 8, 2), (40, 8, 2), (64, 16, 1)])
@pytest.mark.parametrize("where", ["query", "cached key", "cached value", "own key"])
def test_nan_reaches_the_rows_that_see_it(N, Hq, Hkv, where):
    c = Tree(2, N, 300, Hq, Hkv, 128, 64, 0, "chain", seed=24)
    ref = c.reference()
    G = Hq // Hkv
    sees = np.zeros((2, N, Hq), bool)
    if where == "query":
        c.xc[1, 1, 0, 3] = NAN
        sees[1, 1, 0] = True
    elif where == "own key":
        c.kn[1, 1, 0, 3] = NAN
        sees[1, 1:, :G] = True
    else:
        (c.k if where == "cached key" else c.v)[1, 100, 0, 3] = NAN
        sees[1, :, :G] = True
    got = val(c.run()[1])
    if where == "cached value":  # its column of the head dimension
        assert np.isnan(got[1, :, :G, 3]).all()
    else:
        assert np.isnan(got[sees]).all()
    r, bound = ref[1]
    assert_bounded(got[~sees], r[~sees], bound[~sees], "the others")


def test_keys_of_any_size():
    """Cached and own keys of 2^17 and 2^-60 times their size, against queries as much smaller and larger."""
    for e in (17, -60):
        for N in (3, 40):
            c = Tree(1, N, 300, 8, 2, 128, 128, 4, seed=25)
            for arr in (c.k, c.kn):
                arr[(arr & 0x7F80) < (70 << 7)] = 0
                arr[arr != 0] = (arr[arr != 0].astype(np.int32) + (e << 7)).astype(np.uint16)
            for arr in (c.x, c.xc):
                arr[(arr & 0x7F80) < (30 << 7)] = 0
                arr[arr != 0] = (arr[arr != 0].astype(np.int32) - (e << 7)).astype(np.uint16)
            c.vec[1][:], c.vec[3][:] = 0, 0
            err = error_word()
            c.check(c.run(dev_err=err))
            assert int(err.item()) == 0


@pytest.mark.parametrize("N", [2, 40])
def test_bits_do_not_depend_on_workspace_stream_or_graph(N):
    c = Tree(2, N, 3000, 8, 2, 128, 128, 4, ragged=True, seed=26)
    args, nodes = c.args(), i32(c.nodes)
    ref = [torch.zeros_like(args[0]) for _ in range(2)]
    orth.decode_tree(*args, sinks=4, nodes=nodes, o=ref[0], oc=ref[1])
    n = orth.decode_tree_workspace_size(2, N, c.L_max, 8, 2, 128)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev())
    out = [torch.zeros_like(args[0]) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):  # back to back: a call must not start on the one before's partials
            orth.decode_tree(*args, sinks=4, nodes=nodes, o=out[0], oc=out[1], workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(out, ref):
        np.testing.assert_array_equal(bits(a), bits(b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orth.decode_tree(*args, sinks=4, nodes=nodes, o=out[0], oc=out[1], workspace=ws)
    for _ in range(2):
        out[0].zero_(), out[1].zero_(), ws.fill_(0xFF)
        graph.replay()
        for a, b in zip(out, ref):
            np.testing.assert_array_equal(bits(a), bits(b))


def accept_reference(c, node):
    k, v, lens = c.k.copy(), c.v.copy(), c.lens.copy()
    path = np.full(c.parent.shape, -1, np.int32)
    for b, n in enumerate(node):
        if n < 0:
            continue
        way = sink_util.paths(list(c.parent[b]))[n]
        for a, i in enumerate(way):
            path[b, a] = i
            k[b, lens[b] + a], v[b, lens[b] + a] = c.kn[b, i], c.vn[b, i]
        lens[b] += len(way)
    return path, k, v, lens


@pytest.mark.parametrize("B,N,L,Hkv,d,shape", [(1, 1, 0, 1, 64, "chain"), (3, 5, 100, 2, 64, "random"),
                                                (8, 64, 300, 8, 128, "random"), (5, 64, 64, 4, 128, "chain"),
                                                (40, 9, 70, 1, 128, "random"), (2, 33, 10, 3, 64, "star")])
def test_accept(B, N, L, Hkv, d, shape):
    c = Tree(B, N, L, Hkv, Hkv, d, shape=shape, ragged=True, seed=31 + N, room=N)
    rng = np.random.default_rng(N)
    node = rng.integers(-1, N, B).astype(np.int32)
    node[0] = N - 1
    want = accept_reference(c, node)
    k, v, lens, err = bf(c.k), bf(c.v), i32(c.lens), error_word()
    path = orth.decode_tree_accept(bf(c.kn), bf(c.vn), i32(c.parent), i32(node), k, v, lens, dev_err=err)
    np.testing.assert_array_equal(path.cpu().numpy(), want[0])
    np.testing.assert_array_equal(bits(k), want[1])
    np.testing.assert_array_equal(bits(v), want[2])
    np.testing.assert_array_equal(lens.cpu().numpy(), want[3])
    assert int(err.item()) == 0


def test_accept_errors_leave_the_cache_as_it_is():
    c = Tree(6, 4, 50, 2, 2, 64, shape="chain", seed=33)
    c.lens[:] = [10, 10, 10, 48, 47, -3]
    c.parent[2, 1] = 7
    node = np.array([4, -2, 3, 3, 2, 0], np.int32)
    k, v, lens = bf(c.k), bf(c.v), i32(c.lens)
    err = error_word()
    path = orth.decode_tree_accept(bf(c.kn), bf(c.vn), i32(c.parent), i32(node), k, v, lens, dev_err=err)
    assert int(err.item()) == orth.DEVERR_POSITION | orth.DEVERR_CACHE_FULL
    np.testing.assert_array_equal(lens.cpu().numpy(), [10, 10, 10, 48, 50, -3])  # only the fifth fits
    np.testing.assert_array_equal(path.cpu().numpy()[4], [0, 1, 2, -1])
    assert (path.cpu().numpy()[[0, 1, 2, 3, 5]] == -1).all()
    c.k[4, 47:50], c.v[4, 47:50] = c.kn[4, :3], c.vn[4, :3]
    np.testing.assert_array_equal(bits(k), c.k)
    np.testing.assert_array_equal(bits(v), c.v)


@pytest.mark.parametrize("Hq,Hkv,d,sinks", [(8, 2, 128, 0), (8, 2, 64, 4), (32, 8, 128, 4)])
def test_prompt_draft_accept_draft(Hq, Hkv, d, sinks):
    """A prompt through the windowed stream with sinks, then two rounds of drafted chains with acceptance: every
    accepted token's outputs are those of a prompt that holds them all."""
    B, T, n, window = 2, 300, 6, 64
    total = T + 2 * n
    x, xc = (normal_bf16(41, m, (B, total, Hq, d)) for m in ("q_raw", "qc_raw"))
    k, v = (normal_bf16(41, m, (B, total, Hkv, d)) for m in ("k", "v"))
    al, be = scale_offset(41, Hq, d)
    ac, bc = scale_offset(41, Hq, d, prefix="_c")
    ref, bound, _ = sink_util.sink_fwd(f64(x), f64(k), f64(v), al.astype(float), be.astype(float), window, sinks)
    pos = np.tile(np.arange(total, dtype=np.int32), (B, 1))
    refc = oracle.xattn(xc, pos, k, v, ac, bc, d ** -0.5)
    kc, vc = (torch.full((B, total, Hkv, d), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    kc[:, :T], vc[:, :T] = bf(k[:, :T]), bf(v[:, :T])
    o = orth.swa_sink_fwd(bf(x[:, :T]), bf(k[:, :T]), bf(v[:, :T]), f32(al), f32(be), sinks, window=window)
    assert_bounded(val(o), ref[:, :T], bound[:, :T], "prompt")
    lens, at = torch.full((B,), T, dtype=torch.int32, device=dev()), T
    for keep in (4, n):  # the first round's last two are rejected
        parent = i32(parents(None, B, n, "chain"))
        s = slice(at, at + n)
        kn, vn = bf(k[:, s]), bf(v[:, s])
        o, oc = orth.decode_tree(bf(x[:, s]), bf(xc[:, s]), kn, vn, parent, kc, vc, lens, f32(al), f32(be), f32(ac), f32(bc),
                                 window=window, sinks=sinks)
        assert_bounded(val(o), ref[:, s], bound[:, s], "base tokens")
        assert_parity(val(oc), refc[:, s], "copies")
        node = torch.full((B,), keep - 1, dtype=torch.int32, device=dev())
        path = orth.decode_tree_accept(kn, vn, parent, node, kc, vc, lens)
        assert (path[:, :keep] == torch.arange(keep, device=dev())).all() and (path[:, keep:] == -1).all()
        at += keep
        assert (lens == at).all()
        np.testing.assert_array_equal(bits(kc[:, :at]), k[:, :at])
    # and the next single token through the plain decode step, on the cache that the trees left (without sinks)
    if sinks == 0:
        step = slice(at, at + 1)
        o, oc = orth.decode_step(bf(x[:, at]), bf(xc[:, at]), bf(k[:, at]), bf(v[:, at]), kc, vc, lens, f32(al), f32(be),
                                 f32(ac), f32(bc), window=window)
        assert_parity(val(o)[:, None], ref[:, step], "decode step")
        assert_parity(val(oc)[:, None], refc[:, step], "decode step's copies")


@pytest.mark.parametrize("N,Hq", [(1, 8), (7, 32)])
def test_offsets_beyond_32_bits(N, Hq):
    """The third sequence's cache lies behind 2^31 values: as the same sequence alone, and so is what is appended."""
    B, L, L_max, Hkv, d = 3, 400, 1 << 20, 8, 128
    c = Tree(B, N, L, Hq, Hkv, d, sinks=4, seed=41, room=N)
    big = [torch.empty((B, L_max, Hkv, d), dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    for t, small in zip(big, (c.k, c.v)):
        t[:, :L + N] = bf(small)
    a = list(c.args())
    a[5], a[6] = big
    ref = c.run()
    got = orth.decode_tree(*a, window=c.window, sinks=c.sinks)
    c.check(got)
    for y, r in zip(got, ref):
        assert_bounded(val(y), val(r).astype(np.float64), np.abs(val(r)) * 2.0 ** -7 + 1e-2, "as in a small cache")
    node = np.full(B, N - 1, np.int32)
    path, k, v, lens = accept_reference(c, node)
    got = orth.decode_tree_accept(a[2], a[3], a[4], i32(node), *big, a[7])
    np.testing.assert_array_equal(got.cpu().numpy(), path)
    np.testing.assert_array_equal(bits(big[0][:, :L + N]), k)
    np.testing.assert_array_equal(bits(big[1][:, :L + N]), v)
    np.testing.assert_array_equal(a[7].cpu().numpy(), lens)
