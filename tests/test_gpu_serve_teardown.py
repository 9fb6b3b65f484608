"""GPU tests of the shared-prefix kernel where the last 256 query rows of a KV head number at most 128, so that the
second of its two streams has no row: calls behind one another, and others in between, on the same SMs."""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_parity, bits, dev, val
from tests.test_gpu_prefix import Copies, PrefixDecode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T_out,P,T_kv,Hq,Hkv,d", [
    (10, 2, 130, 10, 32, 8, 128),    # one pass, 8 rows a sequence (where it is chosen)
    (6, 65, 300, 50, 32, 8, 128),    # one pass, 260 rows a sequence: 4 in the last tile
    (5, 60, 129, 61, 32, 16, 64),    # one pass, 120 rows: the first tile only
    (33, 10, 600, 40, 8, 8, 128),    # 330 rows of the batch: 74 in the last tile
    (65, 1, 2000, 30, 32, 8, 128),   # one copy a sequence, 260 rows
])
def test_copies_of_a_second_tile_without_rows(B, T_out, P, T_kv, Hq, Hkv, d):
    c = Copies(B, T_out, P, T_kv, Hq, Hkv, d, 800 + T_out)
    other = Copies(4, 150, 200, 40, 32, 8, 128, 900)  # its tiles are full; it takes the SMs over
    ref, ref2 = bits(c.run()), bits(other.run())
    got = [(c.run(), other.run()) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in got:
        np.testing.assert_array_equal(bits(x), ref)
        np.testing.assert_array_equal(bits(y), ref2)
    assert_parity(val(got[-1][0]), c.oracle(), "copies")
    assert_parity(val(got[-1][1]), other.oracle(), "the others")


def test_decode_of_a_second_tile_without_rows():
    lens = tuple(i % 7 for i in range(65))  # 260 rows a KV head
    s = PrefixDecode(lens, 8, 900, 8, 2, 128, 128, 810)
    outs = [s.step(i) for i in range(8)]
    for i in range(8):
        ro, roc = s.oracle_step(i)
        assert_parity(val(outs[i][0]), ro, f"step {i} base")
        assert_parity(val(outs[i][1]), roc, f"step {i} copy")
    assert int(s.err.item()) == 0 and outs[0][0].device == dev()
