"""Host-side refusals of acceptance with each tree's number of nodes (no call here launches anything)."""
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from tests.test_sinks_cpu import L, off, p  # noqa: F401  (fixtures)


def test_accept_nodes_refusals(L, p):  # noqa: F811
    def call(ptrs=None, L_max=64, B=2, N=5, Hkv=2, d=64):
        a = [p] * 8 + [L_max, p]
        for i, v in (ptrs or {}).items():
            a[i] = v
        return L.orthros_decode_tree_accept_nodes(*a, B, N, Hkv, d, None, None)
    for i in [0, 1, 2, 4, 5, 6, 7, 9]:
        assert call({i: None}) == 1, i
    for i in (0, 1, 5, 6):
        assert call({i: off(p, 8)}) == 1, i
        assert call({i: off(p, 8), 3: None}) == 1, i  # without nodes too
    for kw in (dict(B=0), dict(N=0), dict(L_max=0), dict(Hkv=0), dict(B=40000), dict(L_max=2 ** 31 - 10)):
        assert call(**kw) == 1, kw
    for kw in (dict(N=65), dict(d=96)):
        assert call(**kw) == 2, kw


def test_binding_refuses_host_nodes():
    B, N, Hkv, d = 2, 3, 2, 64
    kn, k = (torch.zeros((B, n, Hkv, d), dtype=torch.bfloat16) for n in (N, 16))
    i32 = dict(dtype=torch.int32)
    parent, each = torch.zeros((B, N), **i32), torch.zeros(B, **i32)
    with pytest.raises(orth.OrthrosError):
        orth.decode_tree_accept(kn, kn, parent, each, k, k, each, nodes=each)
