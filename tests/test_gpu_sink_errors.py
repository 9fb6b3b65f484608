"""GPU tests of what the base stream with sinks reports: the error word names what a row's result depends on and
nothing else, and the log-sum-exp of a row that is not a number is none."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from tests.attend_util import assert_bounded
from tests.gpu_util import bf, bits, dev, f32, val
from tests.test_gpu_sinks import Stream, error_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq,Hkv,d,window,sinks", [(8, 2, 128, 128, 4), (8, 4, 64, 77, 1), (16, 1, 128, 33, 31),
                                                   (2, 2, 128, 128, 4), (8, 2, 128, 500, 4)])
def test_keys_behind_the_sinks_that_no_row_sees(Hq, Hkv, d, window, sinks, value):
    """In a range only the sinks themselves have to be in place before its windows: the rows that share their key
    block may hold anything."""
    begin = 640
    s = Stream(2, 900, Hq, Hkv, d, window, sinks, seed=window)
    clean = s.run()
    k = bf(s.k)
    k[:, sinks:32] = value
    err = error_word()
    got = orth.swa_sink_fwd(bf(s.x), k, bf(s.v), f32(s.alpha), f32(s.beta), sinks, window=window, row_begin=begin,
                            dev_err=err)
    np.testing.assert_array_equal(bits(got[:, begin:]), bits(clean[:, begin:]))
    assert int(err.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,d,window,sinks", [(8, 2, 128, 128, 4), (8, 4, 64, 77, 5), (16, 1, 128, 33, 4),
                                                   (8, 2, 128, 128, 0), (2, 2, 128, 128, 4), (8, 2, 128, 500, 4)])
@pytest.mark.parametrize("row", [3, 20, 555])
def test_products_beyond_fp32_that_no_row_sees(Hq, Hkv, d, window, sinks, row):
    """A key of 3e38 in one column and zeros else, against queries that are zero in that column where they see the key
    and 64 where they do not, so that scale log2(e) q.k would be some 3e39: no logit that counts is out of range."""
    s = Stream(1, 1000, Hq, Hkv, d, window, sinks, seed=row)
    t = np.arange(1000)
    seen = (t >= row) & ((t < row + window) | (row < sinks))
    s.alpha[:, 5], s.beta[:, 5] = 1, 0
    s.x[0, :, :, 5] = np.where(seen, 0, 0x4280)[:, None]  # 64
    s.k[0, row] = 0
    s.k[0, row, :, 5] = 0x7F62  # 3.0e38
    ref, bound, _ = s.reference()
    err = error_word()
    got = s.run(dev_err=err)
    assert int(err.item()) == 0
    assert_bounded(val(got), ref, bound, "o")


@pytest.mark.parametrize("T", [500, 60])
@pytest.mark.parametrize("Hq,Hkv,d,window,sinks", [(8, 2, 128, 128, 4), (8, 2, 64, 128, 0), (8, 2, 128, 33, 4),
                                                   (2, 2, 128, 128, 4), (8, 2, 128, 400, 4), (8, 2, 128, 400, 0),
                                                   (2, 2, 64, 128, 0)])
def test_log_sum_exp_of_a_query_that_is_no_number(Hq, Hkv, d, window, sinks, T):
    """Nothing of the buffer is left as it was."""
    s = Stream(2, T, Hq, Hkv, d, window, sinks, seed=T)
    ref, ref_lse = s.run(lse=True)
    at = [(0, 0, 0), (0, T // 2, 1), (1, T - 1, Hq - 1)]
    for b, t, h in at:
        s.x[b, t, h, 7] = 0x7FC0
    lse = torch.full((2, T, Hq), 7.0, device=dev())
    got, _ = s.run(lse=lse)
    row = torch.zeros((2, T, Hq), dtype=torch.bool, device=dev())
    for i in at:
        row[i] = True
    assert torch.isnan(lse[row]).all() and torch.isnan(got.float()[row]).all()
    assert torch.equal(lse[~row], ref_lse[~row]) and torch.equal(got[~row], ref[~row])
    if sinks == 0:
        lse.fill_(7.0)
        orth.swa_fwd_lse(bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), window=window, lse=lse)
        assert torch.isnan(lse[row]).all() and torch.isfinite(lse[~row]).all()
