"""GPU tests of row ranges of the base stream with sinks: a range gives its rows the bits that a call for all rows
gives them, log-sum-exp included, whatever kernel the sizes select for either call."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from tests.gpu_util import bf, bits, dev, f32
from tests.test_gpu_sinks import Stream, error_word

pytestmark = pytest.mark.gpu


def same_as_whole(s, cuts):
    """Each range of cuts alone: its rows as in the whole, no other row written."""
    B, T, Hq, d = s.x.shape
    err = error_word()
    whole, whole_lse = s.run(lse=True, dev_err=err)
    for begin, end in cuts:
        out = torch.full((B, T, Hq, d), 7.0, dtype=torch.bfloat16, device=dev())
        lse = torch.full((B, T, Hq), 7.0, device=dev())
        s.run(out=out, lse=lse, row_begin=begin, row_end=end, dev_err=err)
        np.testing.assert_array_equal(bits(out[:, begin:end]), bits(whole[:, begin:end]), f"{begin} .. {end}")
        assert torch.equal(lse[:, begin:end], whole_lse[:, begin:end]), (begin, end)
        for y in (out, lse):
            assert (y[:, :begin] == 7.0).all() and (y[:, end:] == 7.0).all(), (begin, end)
    assert int(err.item()) == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", [
    (2, 500, 8, 2, 128, 128, 0),    # no sinks, the band in tensor memory
    (1, 400, 8, 4, 64, 128, 0),
    (2, 300, 8, 1, 128, 40, 0),
    (1, 300, 16, 1, 128, 128, 0),
    (1, 140, 16, 1, 64, 140, 4),    # a window over everything leaves nothing to the sinks
    (2, 500, 4, 4, 64, 128, 0),     # ungrouped heads and a wide window
    (1, 600, 8, 2, 128, 500, 0),
])
def test_log_sum_exp_of_a_range_without_sinks(B, T, Hq, Hkv, d, window, sinks):
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + Hq)
    same_as_whole(s, [(0, 128), (128, T)] + ([(128, 256), (256, T)] if T > 256 else []))


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", [
    (1, 5000, 4, 4, 64, 300, 4),     # 160 tiles of 128 tokens, which go by pairs: a range may begin inside a pair
    (2, 2600, 4, 4, 128, 70, 3),
    (1, 2600, 8, 4, 128, 300, 4),    # tiles of 64 tokens
    (1, 1300, 16, 1, 64, 300, 5),    # tiles of 8 tokens
    (3, 1700, 16, 2, 128, 1000, 32),
])
def test_ranges_of_streams_of_many_tiles(B, T, Hq, Hkv, d, window, sinks):
    """More tiles than SMs in the whole, few in the range."""
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + Hkv)
    last = T // 128 * 128
    same_as_whole(s, [(0, 128), (128, 256), (128, 384), (256, 640), (640, 1024), (last, T), (last - 128, T), (384, T)])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks,begin,end", [
    (2, 900, 8, 2, 128, 128, 4, 384, 640),    # the band in tensor memory
    (1, 700, 8, 4, 64, 100, 17, 256, 512),
    (2, 500, 16, 1, 128, 33, 4, 256, 384),
    (2, 900, 8, 2, 128, 128, 0, 384, 640),
    (1, 700, 2, 2, 64, 128, 4, 384, 512),     # tiles of rows
    (1, 5000, 4, 4, 64, 300, 4, 640, 768),
    (1, 1300, 8, 2, 128, 400, 4, 640, 1024),
    (2, 900, 8, 2, 128, 400, 0, 640, 900),    # on warp MMAs
    (1, 700, 2, 2, 64, 120, 0, 384, 512),
    (1, 700, 16, 1, 128, 250, 0, 256, 384),
])
def test_what_a_range_does_not_read(B, T, Hq, Hkv, d, window, sinks, begin, end, value):
    """Keys before the range's first window that are no sinks, and keys, values and queries behind or before the range:
    not in place yet, or not any more."""
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + window)
    whole, whole_lse = s.run(lse=True)
    q, k, v = bf(s.x), bf(s.k), bf(s.v)
    q[:, :begin], q[:, end:] = value, value
    for t in (k, v):
        t[:, sinks:begin - window + 1], t[:, end:] = value, value
    err = error_word()
    o, lse = orth.swa_sink_fwd(q, k, v, f32(s.alpha), f32(s.beta), sinks, window=window, lse=True, row_begin=begin,
                               row_end=end, dev_err=err)
    np.testing.assert_array_equal(bits(o[:, begin:end]), bits(whole[:, begin:end]))
    assert torch.equal(lse[:, begin:end], whole_lse[:, begin:end])
    if sinks == 0:
        o = orth.swa_fwd_rows(q, k, v, f32(s.alpha), f32(s.beta), begin, end, window=window, dev_err=err)
        np.testing.assert_array_equal(bits(o[:, begin:end]), bits(whole[:, begin:end]))
    assert int(err.item()) == 0
