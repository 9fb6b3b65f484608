"""What needs no GPU of the sinks' and trees' entry points: the host-side refusals through the C ABI (none of these
calls launches anything), the workspace sizes, the binding's refusal of host tensors, and the 64-bit references
against differences and closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from tests import sink_util


@pytest.fixture(scope="module")
def L():
    from long_context_attention_orthros_gb300 import build
    build.build()
    return orth.lib()


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * 1024)()
    p = ctypes.c_void_p((ctypes.addressof(buf) + 255) & ~255)  # aligned, never dereferenced
    p.keep = buf
    return p


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_sink_fwd_refusals(L, p):
    def call(ptrs=None, B=1, T=300, Hq=4, Hkv=2, d=128, window=8, sinks=4, scale=0.1, st=(0, 0, 0), rows=(0, 300)):
        a = [p] * 6 + [None]
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_swa_sink_fwd(*a, B, T, Hq, Hkv, d, window, sinks, ctypes.c_float(scale), *st, *rows, None, None)
    for i in range(6):
        assert call({i: None}) == 1 and call({i: off(p, 8)}) == 1, i
    assert call({6: off(p, 4)}) == 1
    for kw in (dict(B=0), dict(T=0), dict(window=0), dict(sinks=-1), dict(scale=float("nan")), dict(st=(3, 0, 0)),
               dict(rows=(0, 301)), dict(rows=(64, 300)), dict(rows=(0, 200)), dict(rows=(-128, 300)),
               dict(rows=(256, 128))):
        assert call(**kw) == 1, kw
    for kw in (dict(sinks=33), dict(d=96), dict(Hq=6, Hkv=4), dict(Hq=96, Hkv=3)):
        assert call(**kw) == 2, kw
    assert call(rows=(128, 128)) == 0  # no row: nothing to do


def test_sink_bwd_refusals(L, p):
    n = L.orthros_swa_sink_bwd_workspace_size(2, 500, 8, 2, 64)
    assert n > L.orthros_swa_bwd_workspace_size(2, 500, 8, 2, 64) > 0
    for a in ((0, 500, 8, 2, 64), (2, 0, 8, 2, 64), (2, 500, 8, 3, 64), (2, 500, 8, 2, 80), (9000, 1, 8, 2, 64)):
        assert L.orthros_swa_sink_bwd_workspace_size(*a) == 0, a

    def call(ptrs=None, B=2, T=500, Hq=8, Hkv=2, d=64, window=128, sinks=4, scale=0.1, ws=p, nbytes=n):
        a = [p] * 13
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_swa_sink_bwd(*a, B, T, Hq, Hkv, d, window, sinks, ctypes.c_float(scale), ws, nbytes, None, None)
    for i in range(13):
        assert call({i: None}) == 1 and call({i: off(p, 4)}) == 1, i
    for kw in (dict(B=0), dict(T=0), dict(window=0), dict(sinks=-1), dict(scale=float("inf")), dict(B=9000)):
        assert call(**kw) == 1, kw
    for kw in (dict(sinks=33), dict(d=32), dict(Hq=7)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(nbytes=n - 1)):
        assert call(**kw) == 3, kw


def test_tree_refusals(L, p):
    n = L.orthros_decode_tree_workspace_size(2, 5, 64, 8, 2, 64)
    assert n > 0
    for a in ((0, 5, 64, 8, 2, 64), (2, 0, 64, 8, 2, 64), (2, 65, 64, 8, 2, 64), (2, 5, 0, 8, 2, 64), (2, 5, 64, 8, 3, 64),
              (2, 5, 64, 8, 2, 96), (40000, 5, 64, 8, 2, 64), (2, 5, 2 ** 31 - 10, 8, 2, 64)):
        assert L.orthros_decode_tree_workspace_size(*a) == 0, a

    def call(ptrs=None, L_max=64, B=2, N=5, Hq=8, Hkv=2, d=64, window=128, sinks=4, scale=0.1, ws=p, nbytes=n):
        a = [p] * 9 + [L_max] + [p] * 6
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_decode_tree(*a, B, N, Hq, Hkv, d, window, sinks, ctypes.c_float(scale), ws, nbytes, None, None)
    for i in [0, 1, 2, 3, 4, 6, 7, 8] + list(range(10, 16)):
        assert call({i: None}) == 1, i
    for i in [0, 1, 2, 3, 6, 7] + list(range(10, 16)):
        assert call({i: off(p, 8)}) == 1, i
    for kw in (dict(B=0), dict(N=0), dict(L_max=0), dict(window=0), dict(sinks=-1), dict(scale=float("nan")), dict(B=40000),
               dict(L_max=2 ** 31 - 10)):
        assert call(**kw) == 1, kw
    for kw in (dict(N=65), dict(sinks=33), dict(d=256), dict(Hq=9)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(nbytes=n - 1), dict(ws=off(p, 16))):
        assert call(**kw) == 3, kw


def test_accept_refusals(L, p):
    def call(ptrs=None, L_max=64, B=2, N=5, Hkv=2, d=64):
        a = [p] * 7 + [L_max, p]
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_decode_tree_accept(*a, B, N, Hkv, d, None, None)
    for i in list(range(7)) + [8]:
        assert call({i: None}) == 1, i
    for i in (0, 1, 4, 5):
        assert call({i: off(p, 8)}) == 1, i
    for kw in (dict(B=0), dict(N=0), dict(L_max=0), dict(Hkv=0)):
        assert call(**kw) == 1, kw
    for kw in (dict(N=65), dict(d=96)):
        assert call(**kw) == 2, kw


def test_binding_refuses_host_tensors():
    B, T, N, Hq, Hkv, d = 1, 16, 3, 4, 2, 64
    bf = dict(dtype=torch.bfloat16)
    x, k, kn = torch.zeros((B, T, Hq, d), **bf), torch.zeros((B, T, Hkv, d), **bf), torch.zeros((B, N, Hkv, d), **bf)
    q, a, lse = torch.zeros((B, N, Hq, d), **bf), torch.zeros((Hq, d)), torch.zeros((B, T, Hq))
    i32 = dict(dtype=torch.int32)
    parent, lens = torch.zeros((B, N), **i32), torch.zeros(B, **i32)
    for f in (lambda: orth.swa_sink_fwd(x, k, k, a, a, 4), lambda: orth.swa_sink_bwd(x, k, k, a, a, x, x, lse, 4),
              lambda: orth.decode_tree(q, q, kn, kn, parent, k, k, lens, a, a, a, a),
              lambda: orth.decode_tree_accept(kn, kn, parent, lens, k, k, lens)):
        with pytest.raises(orth.OrthrosError):
            f()


def test_reference_gradient_against_differences():
    """Central differences of sum(o dO) in 64 bits: truncation some 1e-6 relative at a step of 1e-4."""
    rng = np.random.default_rng(5)
    B, T, Hq, Hkv, d, window, sinks = 1, 14, 2, 1, 4, 3, 2
    x, dO = rng.normal(size=(2, B, T, Hq, d))
    k, v = rng.normal(size=(2, B, T, Hkv, d))
    alpha, beta = 1 + 0.1 * rng.normal(size=(Hq, d)), 0.1 * rng.normal(size=(Hq, d))
    args = [x, k, v, alpha, beta]
    grads = sink_util.sink_bwd(*args, dO, window, sinks)
    for i, g in enumerate(grads):
        step = rng.normal(size=g.shape)
        val = []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * 1e-4 * step
            val.append((sink_util.sink_fwd(*moved, window, sinks)[0] * dO).sum())
        want = (g * step).sum()
        assert abs((val[0] - val[1]) / 2e-4 - want) <= 1e-5 * np.abs(g * step).sum(), i


def test_reference_closed_forms():
    """Equal keys: every row is the mean of the values it sees; a window over everything is causal attention."""
    T, d = 40, 4
    v = np.random.default_rng(6).normal(size=(1, T, 1, d))
    zero, one = np.zeros((1, d)), np.ones((1, d))
    o, _, lse = sink_util.sink_fwd(v * 0, v * 0, v, one, zero, 5, 3)
    for t in range(T):
        rows = sorted(set(range(min(3, t + 1))) | set(range(max(0, t - 4), t + 1)))
        np.testing.assert_allclose(o[0, t, 0], v[0, rows, 0].mean(0), rtol=1e-12)
        np.testing.assert_allclose(lse[0, t, 0], np.log(len(rows)), rtol=1e-12, atol=1e-12)
    assert sink_util.paths([-1, 0, 1, -1, 3, 9, 5]) == [[0], [0, 1], [0, 1, 2], [3], [3, 4], None, None]
