"""GPU tests of the decode step over an 8-bit cache where the sizes of the V rows decide: rows of zeros, rows much
smaller than others that carry no weight, values near the smallest.  Errors are judged against the formula in 64
bits, relative to the output's size."""
import numpy as np
import pytest
import torch

from synthetic import bf16_to_f32
from tests.attend_util import FP16, assert_bounded, attend
from tests.gpu_util import bf, f32, val
from tests.q8_util import code_values, quantize
from tests.test_gpu_kv_q8 import Q8Decode, codes, exps

pytestmark = pytest.mark.gpu


def scaled(bits: np.ndarray, n: int) -> np.ndarray:
    """bf16 bits of x 2^n, for values whose result is normal (those that are smaller become zeros)."""
    ex = (bits.astype(np.int32) >> 7) & 255
    return np.where((ex + n > 0) & (ex > 0), bits.astype(np.int32) + (n << 7), 0).astype(np.uint16)


class Step:
    """A decode step whose K and V rows the test sets (bf16 bits) before they are quantised."""

    def __init__(self, lens, Hq, Hkv, d, code, seed, window=128):
        self.s = Q8Decode(lens, 1, Hq, Hkv, d, window, code, seed)
        n = self.s.inp
        self.k, self.v = (x[:, :max(lens)].copy() for x in (n.k_cache, n.v_cache))
        self.code, self.lens = code, lens

    def check(self, what=""):
        s, n = self.s, self.s.inp
        for j, rows in enumerate((self.k, self.v)):
            for b, m in enumerate(self.lens):
                s.codes[j][b, :m], s.exps[j][b, :m] = quantize(rows[b, :m], self.code)
        s.dev_cache = [codes(c, self.code) for c in s.codes] + [exps(e) for e in s.exps]
        s.vec = [f32(x) for x in (n.alpha, n.beta, n.alpha_c, n.beta_c)]
        o, oc = (val(x) for x in s.step(0))
        cfg = s.cfg
        G = cfg.Hq // cfg.Hkv
        new = [quantize(x, self.code) for x in (n.k_new[0], n.v_new[0])]
        for b, m in enumerate(self.lens):
            for g in range(cfg.Hkv):
                k, v = (np.concatenate([code_values(s.codes[j][b, :m, g], self.code) *
                                        np.exp2(s.exps[j][b, :m, g].astype(float))[:, None],
                                        (code_values(new[j][0][b, g], self.code) * 2.0 ** float(new[j][1][b, g]))[None]])
                        for j in range(2))
                h = slice(g * G, (g + 1) * G)
                for name, got, x, al, be, first in (("base", o, n.q_new, n.alpha, n.beta, max(0, m + 1 - cfg.window)),
                                                    ("copy", oc, n.qc_new, n.alpha_c, n.beta_c, 0)):
                    q = (bf16_to_f32(x[0][b, h]).astype(np.float64) * al[h] + be[h]) * cfg.scale
                    # the query and the probabilities are rounded to fp16
                    ref, bound = attend(q, k[first:], v[first:], FP16, FP16)
                    assert_bounded(got[b, h], ref, bound, f"{what} {name} {b} {g}")
        torch.cuda.synchronize()
        assert int(s.err.item()) == 0


SHAPES = [((400,), 8, 2, 64), ((1300, 65), 32, 8, 128), ((333,), 4, 4, 128), ((517,), 16, 1, 128), ((300,), 16, 2, 64)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,Hq,Hkv,d", SHAPES)
def test_values_near_the_smallest(lens, Hq, Hkv, d, code):
    """Every V row is so small that its exponent is near -126, the new one too."""
    t = Step(lens, Hq, Hkv, d, code, 71)
    n = -119 if code == "e4m3" else -121
    t.v, t.s.inp.v_new[0] = scaled(t.v, n), scaled(t.s.inp.v_new[0], n)
    assert quantize(t.v, code)[1].min() < -120
    t.check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("shift", [-10, -17, -24, -60])
@pytest.mark.parametrize("lens,Hq,Hkv,d", SHAPES)
def test_rows_of_zeros_among_small_values(lens, Hq, Hkv, d, shift, code):
    """A row of zeros (its exponent is 0, above all others) takes weight but no other row's bits, wherever it lies:
    first, in a block's middle, in the window, as the new token."""
    t = Step(lens, Hq, Hkv, d, code, 72)
    t.v, t.s.inp.v_new[0] = scaled(t.v, shift), scaled(t.s.inp.v_new[0], shift)
    for b, m in enumerate(lens):
        t.v[b, [0, 40, m - 60, m - 1]] = 0
        t.v[b, m // 2] = 0x8000  # zeros of the other sign
    t.check("rows")
    t = Step(lens, Hq, Hkv, d, code, 73)
    t.v, t.s.inp.v_new[0] = scaled(t.v, shift), 0
    t.check("new row")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,Hq,Hkv,d", SHAPES)
def test_every_value_is_zero(lens, Hq, Hkv, d, code):
    t = Step(lens, Hq, Hkv, d, code, 74)
    t.v[:], t.s.inp.v_new[0] = 0, 0
    s = t.s
    for j, rows in enumerate((t.k, t.v)):
        for b, m in enumerate(lens):
            s.codes[j][b, :m], s.exps[j][b, :m] = quantize(rows[b, :m], code)
    s.dev_cache = [codes(c, code) for c in s.codes] + [exps(e) for e in s.exps]
    o, oc = s.step(0)
    assert not o.any() and not oc.any() and int(s.err.item()) == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("shift", [-17, -60, -100])
@pytest.mark.parametrize("lens,Hq,Hkv,d", SHAPES)
def test_large_values_without_weight(lens, Hq, Hkv, d, shift, code):
    """V rows of ordinary size whose keys every query avoids (weights under 2^-80), among rows smaller by 2^shift."""
    t = Step(lens, Hq, Hkv, d, code, 75)
    n = t.s.inp
    far = 64 if shift > -80 else 128  # nats below the others
    for al, be in ((n.alpha, n.beta), (n.alpha_c, n.beta_c)):
        al[:, 0], be[:, 0] = 0, far / 8 / t.s.cfg.scale  # column 0 of every scaled query is far / 8
    small = scaled(t.v, shift)
    t.k[..., 0] = 0
    n.k_new[0][..., 0] = 0
    n.v_new[0] = scaled(n.v_new[0], shift)
    for b, m in enumerate(lens):
        for r in (3, m // 2, m - 30):
            small[b, r] = t.v[b, r]
            t.k[b, r], t.k[b, r, :, 0] = 0, 0xC100  # -8
    t.v = small
    t.check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,Hq,Hkv,d", SHAPES)
def test_large_values_of_little_weight(lens, Hq, Hkv, d, code):
    """V rows whose sizes span 2^-50 .. 2^50, their weights the other way round: all count in the output alike."""
    t = Step(lens, Hq, Hkv, d, code, 76)
    n = t.s.inp
    for al, be in ((n.alpha, n.beta), (n.alpha_c, n.beta_c)):
        al[:, 0], be[:, 0] = 0, 4 / t.s.cfg.scale  # column 0 of every scaled query is 4
    t.k[..., 0], n.k_new[0][..., 0] = 0, 0
    rng = np.random.default_rng(77)
    for b, m in enumerate(lens):
        for r in range(m):
            size = int(rng.integers(-50, 51))
            t.v[b, r] = scaled(t.v[b, r], size)
            t.k[b, r, :, 0] = np.float32(-size * np.log(2) / 4).view(np.uint32) >> 16
    t.check()
