"""How the binding reads batch strides: the library takes 0 for the dense stride, so a batch expanded from one
sequence (stride 0) must be refused, not read past its end.  The checks run without a GPU on stand-ins that report a device; the public calls
refuse on one."""
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from long_context_attention_orthros_gb300 import _binding


class OnDevice:
    """A host tensor that says it is on device 0; only its shape, strides and type are read."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self._t, name)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("T", [1, 7])
def test_expanded_batches_are_refused(T):
    x = OnDevice(bf(1, T, 2, 64).expand(3, -1, -1, -1))
    with pytest.raises(orth.OrthrosError):
        _binding._bf16_rows(x, "x")
    with pytest.raises(orth.OrthrosError):
        _binding._rows(x, "x", x.shape, 0)
    with pytest.raises(orth.OrthrosError):
        _binding._kv_pair(x, x, 3, 2, 64, 0)


def test_other_batch_strides_are_read_as_they_are():
    dense, longer = bf(3, 7, 2, 64), bf(3, 9, 2, 64)[:, :7]
    assert _binding._bf16_rows(OnDevice(dense), "x") == 7 * 128
    assert _binding._bf16_rows(OnDevice(longer), "x") == 9 * 128
    assert _binding._rows(OnDevice(dense), "x", dense.shape, 0)[1] == 0
    assert _binding._rows(OnDevice(longer), "x", longer.shape, 0)[1] == 9 * 128
    one = bf(1, 7, 2, 64)
    assert _binding._bf16_rows(OnDevice(one.expand(1, -1, -1, -1)), "x") == 7 * 128
    assert _binding._bf16_rows(OnDevice(one[:, :5]), "x") == 5 * 128
    assert _binding._bf16_rows(OnDevice(bf(1, 0, 2, 64).expand(3, -1, -1, -1)), "x") in (0, 128)  # no row is read


@pytest.mark.gpu
def test_public_calls_refuse_expanded_tensors():
    B, T, Hq, Hkv, d = 3, 5, 4, 2, 64
    dev = torch.device("cuda:0")

    def z(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=dev)
    rows, wide, q = z(B, T, Hkv, d), z(1, T, Hkv, d).expand(B, -1, -1, -1), z(B, 1, Hq, d)
    wide_q = z(1, 1, Hq, d).expand(B, -1, -1, -1)
    cache = orth.kv_cache_q8(B, 16, Hkv, d, dev)
    pre, pos = z(9, Hkv, d), torch.zeros((B, 1), dtype=torch.int32, device=dev)
    a = torch.zeros((Hq, d), device=dev)
    for call in (lambda: orth.kv_quantize(wide, wide, *cache), lambda: orth.kv_dequantize(*cache, wide, wide),
                 lambda: orth.xattn_prefix_fwd(wide_q, pos, pre, pre, rows, rows, a, a),
                 lambda: orth.xattn_prefix_fwd(q, pos, pre, pre, wide, wide, a, a),
                 lambda: orth.xattn_prefix_fwd(q, pos, pre, pre, rows, rows, a, a, out=wide_q),
                 lambda: orth.xattn_fwd(wide_q, pos, rows, rows, a, a), lambda: orth.xattn_fwd(q, pos, wide, wide, a, a),
                 lambda: orth.swa_fwd(z(B, T, Hq, d), wide, wide, a, a)):
        with pytest.raises(orth.OrthrosError):
            call()
