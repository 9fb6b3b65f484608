"""GPU tests of the log-sum-exp that the base stream with sinks writes where a row sees more than 64 keys: q is rounded
to fp16 once, and nothing else is allowed for but 32-bit arithmetic."""
import numpy as np
import pytest

from synthetic import bf16_bits
from tests import sink_util
from tests.test_gpu_sinks import Stream, error_word, f64

pytestmark = pytest.mark.gpu


def bounds(s):
    """Each row's log-sum-exp in 64 bits, what the kernel's may be off at most, and in root mean square [B, T, Hq].

    A rounding moves q_i by at most 2^-11 of itself, with a root mean square of 2^-11 / sqrt(3), and the same q enters
    all logits of a row.  So the log-sum-exp moves by sum_i dq_i kbar_i, kbar the keys' mean by the row's weights, and
    in second order by half the weights' variance of the logits' errors, at most (2^-11 max_j sum_i |q_i k_ji|)^2 / 2.
    32 bits: a logit's sum of d products is truncated at each of d / 16 steps, 8 2^-22 of its products' sizes at most;
    exponentials (2^-22 each), their sum of up to 1032 terms in four parts or more (260 roundings of 2^-24) and its
    logarithm (2^-21) come to less than 2^-15."""
    B, T, Hq, d = s.x.shape
    k, G = f64(s.k), Hq // s.k.shape[2]
    seen = sink_util.sink_seen(T, s.window, s.sinks)
    lse, most, rms = (np.empty((B, T, Hq)) for _ in range(3))
    for b in range(B):
        for h in range(Hq):
            kk = k[b, :, h // G]
            q = (f64(s.x[b, :, h]) * s.alpha[h].astype(np.float64) + s.beta[h]) * d ** -0.5
            x = np.where(seen, q @ kk.T, -np.inf)
            m = x.max(-1, keepdims=True)
            w = np.exp(x - m)
            lse[b, :, h] = (m + np.log(w.sum(-1, keepdims=True)))[:, 0]
            kbar = w @ kk / w.sum(-1, keepdims=True)
            size = np.where(seen, np.abs(q) @ np.abs(kk).T, 0).max(-1)
            rest = (2.0 ** -11 * size) ** 2 / 2 + 8 * 2.0 ** -22 * size
            most[b, :, h] = 2.0 ** -11 * np.abs(q * kbar).sum(-1) + rest + 2.0 ** -15
            rms[b, :, h] = 2.0 ** -11 / 3 ** 0.5 * np.sqrt(((q * kbar) ** 2).sum(-1)) + rest + 2.0 ** -15
    return lse, most, rms


CASES = [
    (2, 500, 8, 2, 128, 128, 4),    # the band in tensor memory
    (1, 500, 8, 4, 64, 128, 17),
    (1, 400, 16, 1, 128, 100, 4),
    (1, 500, 8, 1, 64, 70, 32),
    (2, 500, 2, 2, 128, 128, 4),    # tiles of rows
    (1, 1300, 8, 2, 64, 1000, 32),
    (1, 700, 4, 4, 64, 300, 4),
]


def check(s, independent):
    """independent: every row's roundings are its own."""
    ref, most, rms = bounds(s)
    err = error_word()
    _, lse = s.run(lse=True, dev_err=err)
    off = np.abs(lse.cpu().numpy() - ref)
    assert int(err.item()) == 0
    assert (off <= most).all(), (off / most).max()
    if independent:  # thousands of rows: their mean square comes to its expectation
        many = off[:, 64:]
        assert np.sqrt((many ** 2).mean()) <= 1.25 * np.sqrt((rms[:, 64:] ** 2).mean())


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", CASES)
def test_many_keys(B, T, Hq, Hkv, d, window, sinks):
    check(Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + d), True)


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", CASES)
def test_all_weight_on_one_sink(B, T, Hq, Hkv, d, window, sinks):
    """The queries lie along the first key, whose logit is some 40 then: nothing evens out, and the rows of a head share
    their roundings."""
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + d + 1)
    first = s.k[:, :1].repeat(Hq // Hkv, 2)  # [B, 1, Hq, d]
    k = f64(first)
    c = 40 * d ** 0.5 / (k ** 2).sum(-1, keepdims=True)
    s.x[:] = bf16_bits(np.broadcast_to(k * c, s.x.shape).astype(np.float32).ravel()).reshape(s.x.shape)
    s.alpha[:], s.beta[:] = 1 + 2.0 ** -7 * np.linspace(-1, 1, d), 0  # products that fp16 does not hold
    check(s, False)
