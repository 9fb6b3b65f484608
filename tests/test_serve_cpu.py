"""What needs no GPU of the 8-bit cache and shared-prefix entry points: the host-side refusals through the C ABI
(none of these calls launches anything), the workspace sizes, and the binding's refusal of host tensors."""
import ctypes

import pytest
import torch

import long_context_attention_orthros_gb300 as orth


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


@pytest.mark.parametrize("name", ["orthros_kv_quantize", "orthros_kv_dequantize"])
def test_quantize_refusals(L, p, name):
    def call(ptrs=None, B=2, T=10, Hkv=2, d=64, L_max=32, code=0, stride=0):
        a = [p, p, None, None, p, p, p, p] if name.endswith("kv_quantize") else [p, p, p, p, None, None, p, p]
        for i, v in (ptrs or {}).items():
            a[i] = v
        return getattr(L, name)(*a, B, T, Hkv, d, L_max, code, stride, None, None)
    needed = [0, 1, 4, 5, 6, 7] if name.endswith("kv_quantize") else [0, 1, 2, 3, 6, 7]
    for i in needed:
        assert call({i: None}) == 1 and call({i: off(p, 8)}) == 1
    for kw in (dict(B=0), dict(T=-1), dict(Hkv=0), dict(L_max=0), dict(L_max=40), dict(stride=3), dict(stride=8)):
        assert call(**kw) == 1, kw
    for kw in (dict(d=96), dict(code=2), dict(code=-1)):
        assert call(**kw) == 2, kw
    assert call(T=0) == 0  # nothing to write


def test_decode_q8_refusals(L, p):
    n = L.orthros_decode_q8_workspace_size(2, 64, 8, 2, 64)
    assert n > 0
    for a in ((0, 64, 8, 2, 64), (2, 0, 8, 2, 64), (2, 60, 8, 2, 64), (2, 64, 6, 4, 64), (2, 64, 8, 2, 80),
              (40000, 64, 8, 2, 64)):
        assert L.orthros_decode_q8_workspace_size(*a) == 0, a

    def call(ptrs=None, L_max=64, code=0, B=2, Hq=8, Hkv=2, d=64, window=128, scale=0.1, ws=p, nbytes=n):
        a = [p] * 9 + [L_max, code] + [p] * 6
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_decode_step_q8(*a, B, Hq, Hkv, d, window, ctypes.c_float(scale), ws, nbytes, None, None)
    for i in list(range(9)) + list(range(11, 17)):
        assert call({i: None}) == 1, i
    for i in list(range(8)) + list(range(11, 17)):
        assert call({i: off(p, 4)}) == 1, i
    for kw in (dict(B=0), dict(L_max=0), dict(L_max=72), dict(window=0), dict(scale=float("inf")), dict(B=40000)):
        assert call(**kw) == 1, kw
    for kw in (dict(d=32), dict(Hq=96, Hkv=3), dict(Hq=7), dict(code=5)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(nbytes=n - 1), dict(ws=off(p, 16))):
        assert call(**kw) == 3, kw


def test_decode_prefix_refusals(L, p):
    n = L.orthros_decode_prefix_workspace_size(2, 100, 64, 8, 2, 64)
    assert n > 0
    for a in ((2, 0, 64, 8, 2, 64), (2, 100, 0, 8, 2, 64), (2, 2 ** 31 - 10, 64, 8, 2, 64), (2, 100, 64, 8, 3, 64)):
        assert L.orthros_decode_prefix_workspace_size(*a) == 0, a

    def call(ptrs=None, P=100, L_max=64, B=2, Hq=8, Hkv=2, d=64, window=128, scale=0.1, ws=p, nbytes=n):
        a = [p] * 6 + [P] + [p] * 3 + [L_max] + [p] * 6
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_decode_step_prefix(*a, B, Hq, Hkv, d, window, ctypes.c_float(scale), ws, nbytes, None, None)
    for i in list(range(6)) + [7, 8, 9] + list(range(11, 17)):
        assert call({i: None}) == 1, i
    for kw in (dict(P=0), dict(B=0), dict(L_max=0), dict(window=0), dict(scale=float("nan")), dict(P=2 ** 31 - 10)):
        assert call(**kw) == 1, kw
    for kw in (dict(d=256), dict(Hq=9)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(nbytes=n - 1), dict(ws=off(p, 16))):
        assert call(**kw) == 3, kw


def test_xattn_prefix_refusals(L, p):
    n = L.orthros_xattn_prefix_workspace_size(2, 3, 100, 64, 8, 2, 64)
    assert n > 0
    assert L.orthros_xattn_prefix_workspace_size(2, 0, 100, 64, 8, 2, 64) == 256
    for a in ((2, -1, 100, 64, 8, 2, 64), (2, 3, 0, 64, 8, 2, 64), (2, 3, 100, 0, 8, 2, 64), (2, 3, 100, 64, 8, 3, 64)):
        assert L.orthros_xattn_prefix_workspace_size(*a) == 0, a

    def call(ptrs=None, P=100, B=2, T_out=3, T_kv=64, Hq=8, Hkv=2, d=64, scale=0.1, st=(0, 0, 0), ws=p, nbytes=n):
        a = [p] * 4 + [P] + [p] * 5
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_xattn_prefix_fwd(*a, B, T_out, T_kv, Hq, Hkv, d, ctypes.c_float(scale), *st, ws, nbytes, None,
                                          None)
    for i in (0, 1, 2, 3, 5, 6, 7, 8, 9):
        assert call({i: None}) == 1, i
    for kw in (dict(P=0), dict(B=0), dict(T_out=-1), dict(T_kv=0), dict(scale=float("nan")), dict(st=(8, 0, 0)),
               dict(st=(0, 2 ** 20 + 1, 0)), dict(st=(0, 0, 16))):
        assert call(**kw) == 1, kw
    for kw in (dict(d=96), dict(Hq=9), dict(Hq=64, Hkv=2)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(nbytes=n - 1), dict(ws=off(p, 16))):
        assert call(**kw) == 3, kw
    assert call(T_out=0, ws=None) == 0


def test_binding_refuses_host_tensors_and_wrong_caches():
    B, T, Hq, Hkv, d = 1, 16, 4, 2, 64
    bf = dict(dtype=torch.bfloat16)
    cache = orth.kv_cache_q8(B, T - 3, Hkv, d, "cpu")
    assert cache[0].shape == (B, 16, Hkv, d) and cache[2].shape == (B, Hkv, 16)
    assert orth.kv_cache_q8(B, T, Hkv, d, "cpu", dtype=torch.int8)[0].dtype == torch.int8
    with pytest.raises(orth.OrthrosError):
        orth.kv_cache_q8(B, T, Hkv, d, "cpu", dtype=torch.uint8)
    k, q, n = torch.zeros((B, T, Hkv, d), **bf), torch.zeros((B, Hq, d), **bf), torch.zeros((B, Hkv, d), **bf)
    a, cl = torch.zeros((Hq, d)), torch.zeros(B, dtype=torch.int32)
    pre = torch.zeros((5, Hkv, d), **bf)
    for f in (lambda: orth.kv_quantize(k, k, *cache), lambda: orth.kv_dequantize(*cache, k, k),
              lambda: orth.decode_step_q8(q, q, n, n, *cache, cl, a, a, a, a),
              lambda: orth.decode_step_prefix(q, q, n, n, pre, pre, k, k, cl, a, a, a, a),
              lambda: orth.xattn_prefix_fwd(q[:, None], cl[:, None], pre, pre, k, k, a, a)):
        with pytest.raises(orth.OrthrosError):
            f()
