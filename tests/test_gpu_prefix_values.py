"""GPU tests of the attention behind a shared prefix where keys are small and queries as much larger: the logits are
those of ordinary sizes, whatever the number of query rows a KV head (which chooses the kernel).  Errors are judged
against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from synthetic import bf16_to_f32
from tests.attend_util import BF16, FP16, assert_bounded, attend
from tests.gpu_util import assert_parity, bf, f32, val
from tests.test_gpu_prefix import Copies, PrefixDecode, error_word
from tests.test_gpu_q8_values import scaled

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 8, 2, 64), (4, 1, 8, 2, 128), (16, 1, 8, 1, 128), (40, 1, 8, 1, 128), (40, 1, 16, 4, 64), (300, 1, 4, 1, 128),
          (9, 7, 8, 2, 128), (33, 9, 4, 4, 64), (10, 64, 32, 8, 128), (5, 60, 64, 8, 64), (7, 48, 64, 4, 128)]


def values(bits):
    return bf16_to_f32(bits).astype(np.float64)


def check(c, got, err):
    G = c.qc.shape[2] // c.k.shape[2]
    for b in range(0, len(c.k), max(1, len(c.k) // 5)):
        for g in range(0, c.k.shape[2], 3):
            h = slice(g * G, (g + 1) * G)
            for i in range(0, c.qc.shape[1], 11):
                n = c.pos[b, i] + 1
                k, v = (values(np.concatenate([p[:, g], x[b, :n, g]])) for p, x in ((c.kp, c.k), (c.vp, c.v)))
                q = (values(c.qc[b, i, h]) * c.ac[h] + c.bc[h]) * c.scale
                # queries as fp16 (with a bf16 residual elsewhere, which is finer); probabilities as bf16, twice where
                # the maximum rises inside a pair of blocks
                ref, bound = attend(q, k, v, FP16, 2 * BF16)
                assert_bounded(got[b, i, h], ref, bound, f"{b} {i} {g}")
    assert int(err.item()) == 0


@pytest.mark.parametrize("shift", [12, 17, 24, 60])
@pytest.mark.parametrize("B,T_out,Hq,Hkv,d", SHAPES)
def test_small_keys_and_large_queries(B, T_out, Hq, Hkv, d, shift):
    c = Copies(B, T_out, 333, 70, Hq, Hkv, d, 28)
    c.kp, c.k = scaled(c.kp, -shift), scaled(c.k, -shift)
    c.ac, c.bc = (x * np.float32(2.0 ** shift) for x in (c.ac, c.bc))
    err = error_word()
    check(c, val(c.run(dev_err=err)), err)


@pytest.mark.parametrize("B,T_out,Hq,Hkv,d", SHAPES)
def test_small_ordinary_large_and_zero_keys_together(B, T_out, Hq, Hkv, d):
    """Key rows of sizes 2^-60 .. 2^18 with one column a row, against queries that are as large as each needs."""
    c = Copies(B, T_out, 333, 70, Hq, Hkv, d, 29)
    sizes = np.array([-60, -30, -18, -13, -9, 0, 3, 18, None], dtype=object)
    rng = np.random.default_rng(30)
    c.ac[:], c.bc[:] = 1, 0
    keep = c.qc.copy()
    c.qc[:] = 0
    for col, size in enumerate(sizes[:-1]):
        c.qc[..., col] = scaled(keep[..., col], 3 - int(size))
    for x in (c.kp.reshape(-1, Hkv, d), c.k.reshape(-1, Hkv, d)):
        for r in range(len(x)):
            for g in range(Hkv):
                col = int(rng.integers(0, len(sizes)))
                one = x[r, g, col]
                x[r, g] = 0
                if sizes[col] is not None:
                    x[r, g, col] = scaled(one, int(sizes[col]))
    # a query row spans 2^78 of size, which fp16 with one factor a row cannot hold: each copy looks at one size
    look = rng.integers(0, len(sizes) - 1, c.qc.shape[:3])
    c.qc[np.arange(d) != look[..., None]] = 0
    err = error_word()
    check(c, val(c.run(dev_err=err)), err)


@pytest.mark.parametrize("B", [2, 20, 40])
def test_decode_with_small_keys_and_large_queries(B):
    t = PrefixDecode(tuple(range(B)), 1, 500, 8, 2, 128, 128, 31)
    t.kp, t.k = scaled(t.kp, -24), np.where(t.k == 0x7FC0, t.k, scaled(t.k, -24))
    t.inp.k_new[0] = scaled(t.inp.k_new[0], -24)
    t.dk, t.dkp = bf(t.k[:, t.P:]), bf(t.kp)
    for name in ("alpha", "beta", "alpha_c", "beta_c"):
        getattr(t.inp, name)[...] *= np.float32(2.0 ** 24)
    t.vec = [f32(x) for x in (t.inp.alpha, t.inp.beta, t.inp.alpha_c, t.inp.beta_c)]
    o, oc = t.step(0)
    ro, roc = t.oracle_step(0)
    assert_parity(val(o), ro, "base")
    assert_parity(val(oc), roc, "copy")
    torch.cuda.synchronize()
    assert int(t.err.item()) == 0
