"""GPU tests of what copies behind a shared prefix must not be told: own rows that no copy has reached may hold
anything, and a key that some copies do not see yet is none of theirs.  The error word stays clear on every path."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from tests.gpu_util import assert_parity, bf, f32, i32, val
from tests.test_gpu_prefix import Copies, error_word

pytestmark = pytest.mark.gpu

SHAPES = [(10, 64, 32, 8, 130), (10, 64, 32, 8, 64), (7, 48, 64, 4, 1), (5, 60, 64, 8, 61), (3, 1, 8, 2, 100),
          (40, 1, 8, 1, 65), (2, 2, 8, 2, 101), (3, 3, 8, 2, 70), (1, 30, 8, 2, 17)]


@pytest.mark.parametrize("rest", [0x7F80, 0xFF80, 0x7F62, 0x7FC0], ids=["inf", "-inf", "3e38", "nan"])
@pytest.mark.parametrize("B,T_out,Hq,Hkv,used", SHAPES)
def test_rows_behind_the_last_position_report_nothing(B, T_out, Hq, Hkv, used, rest):
    c = Copies(B, T_out, 200, 300, Hq, Hkv, 128, 24)
    c.pos = np.minimum(c.pos, used - 1)
    c.pos[:, 0] = used - 1
    k, v = c.k.copy(), c.v.copy()
    k[:, used:], v[:, used:] = rest, rest
    err = error_word()
    got = orth.xattn_prefix_fwd(bf(c.qc), i32(c.pos), bf(c.kp), bf(c.vp), bf(k), bf(v), f32(c.ac), f32(c.bc),
                                scale=c.scale, dev_err=err)
    assert_parity(val(got), c.oracle(), "copies")
    assert int(err.item()) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T_out,Hq,Hkv", [(10, 64, 32, 8), (3, 3, 8, 2), (6, 65, 32, 8)])
def test_a_key_behind_some_copies_is_not_theirs(B, T_out, Hq, Hkv, d):
    """Own row 40 holds one huge value: the logits of the copies that see it are 0 (their queries are 0 there), those
    of the copies before it would pass fp32's range."""
    c = Copies(B, T_out, 200, 300, Hq, Hkv, d, 26)
    c.pos[:, 0] = 7
    c.k[:, 40] = 0
    c.k[:, 40, :, 5] = 0x7F00  # 2^127
    c.ac[:, 5], c.bc[:, 5] = 1, 0
    c.qc[..., 5] = np.where(c.pos >= 40, 0, 0x4280)[..., None]  # 64
    err = error_word()
    got = c.run(dev_err=err)
    assert_parity(val(got), c.oracle(), "copies")
    assert int(err.item()) == 0


@pytest.mark.parametrize("where,rows", [("prefix", 40), ("prefix", -1), ("own", -1)])
def test_infinite_keys_that_copies_see_are_reported(where, rows):
    """The error that must stay: an infinite key among the rows that count, where a kernel takes keys as fp16."""
    B, T_out, Hq, Hkv = (10, 64, 32, 8) if rows < 0 else (rows, 1, 8, 1)
    c = Copies(B, T_out, 300, 100, Hq, Hkv, 128, 27)
    (c.kp if where == "prefix" else c.k)[..., 20, 0, 3] = 0x7F80
    err = error_word()
    c.run(dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == orth.DEVERR_RANGE
