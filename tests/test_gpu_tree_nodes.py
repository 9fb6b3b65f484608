"""GPU tests of trees with fewer nodes than the batch's largest: acceptance knows each tree's size, and no error
reaches the rows behind a tree."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from tests.gpu_util import bf, bits, dev, i32, val
from tests.test_gpu_tree import Tree, accept_reference, error_word

pytestmark = pytest.mark.gpu


def test_accept_refuses_nodes_behind_a_tree():
    """A node that is none of its tree's leaves the cache as it is, and so does a number of nodes out of range; what
    lies behind a tree (here parents that are none) does not matter."""
    c = Tree(7, 8, 60, 2, 2, 64, seed=35, room=8)
    nodes = np.array([8, 3, 3, 0, 9, -1, 0], np.int32)
    node = np.array([7, 2, 3, 0, 1, -1, -1], np.int32)
    c.parent[1, 3:], c.parent[2, 3:] = 99, 99
    k, v, lens, err = bf(c.k), bf(c.v), i32(c.lens), error_word()
    path = orth.decode_tree_accept(bf(c.kn), bf(c.vn), i32(c.parent), i32(node), k, v, lens, dev_err=err, nodes=i32(nodes))
    want = accept_reference(c, np.array([7, 2, -1, -1, -1, -1, -1], np.int32))
    np.testing.assert_array_equal(path.cpu().numpy(), want[0])
    np.testing.assert_array_equal(bits(k), want[1])
    np.testing.assert_array_equal(bits(v), want[2])
    np.testing.assert_array_equal(lens.cpu().numpy(), want[3])
    assert int(err.item()) == orth.DEVERR_POSITION


@pytest.mark.parametrize("N,d", [(1, 64), (9, 128), (64, 64)])
def test_accept_with_nodes(N, d):
    """Every node of every tree is accepted as without nodes, and reports nothing."""
    c = Tree(12, N, 100, 2, 2, d, ragged=True, seed=36 + N, room=N)
    rng = np.random.default_rng(N)
    node = (rng.integers(-1, 10 ** 6, 12) % (c.nodes + 1) - 1).astype(np.int32)
    k, v, lens, err = bf(c.k), bf(c.v), i32(c.lens), error_word()
    path = orth.decode_tree_accept(bf(c.kn), bf(c.vn), i32(c.parent), i32(node), k, v, lens, dev_err=err, nodes=i32(c.nodes))
    want = accept_reference(c, node)
    np.testing.assert_array_equal(path.cpu().numpy(), want[0])
    np.testing.assert_array_equal(bits(k), want[1])
    np.testing.assert_array_equal(bits(v), want[2])
    np.testing.assert_array_equal(lens.cpu().numpy(), want[3])
    assert int(err.item()) == 0


@pytest.mark.parametrize("N,Hq,Hkv", [(2, 8, 2), (20, 8, 2), (64, 8, 1)])
def test_a_bad_length_writes_no_row_behind_a_tree(N, Hq, Hkv):
    """Zeros for the tree's nodes, the error bit for a tree without any too, and every row behind them as it was."""
    c = Tree(5, N, 200, Hq, Hkv, 64, sinks=4, seed=37)
    c.nodes = np.array([N - 1, N // 2, 0, N, 0], np.int32)
    for lens in ([-1, 201, 200, 201, 200], [200, 200, 201, 200, -5]):
        c.lens[:] = lens
        o, oc = (torch.full((5, N, Hq, 64), 5.0, dtype=torch.bfloat16, device=dev()) for _ in range(2))
        err = error_word()
        got = [val(y) for y in c.run(o=o, oc=oc, dev_err=err)]
        assert int(err.item()) == orth.DEVERR_CACHE_FULL
        for y in got:
            for b in range(5):
                n = c.nodes[b]
                assert (y[b, n:] == 5).all(), b
                assert (y[b, :n] == 0).all() if not 0 <= lens[b] <= 200 else y[b, :n].any() or n == 0, b
