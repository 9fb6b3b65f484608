"""Plain attention of a few query rows in 64 bits, with a bound on what a kernel's roundings may add.

A logit's error is at most r |q| . |k| (the query rounded by a relative r of its values); weights change by their
logit's error less the weighted mean of all, so the output by at most
    sum_j w_j |v_j| (D_j + sum_i w_i D_i),   D_j = r |q| . |k_j|.
Probabilities rounded by a relative p add p sum_j w_j |v_j|, and the output's own rounding to bf16 half a step,
2^-8 |o|.  32-bit sums, exponentials and products are counted as 2^-12 sum_j w_j |v_j| together (2^-23 each, over a
few thousand keys), second-order terms as a tenth of the first."""
import numpy as np

BF16, FP16 = 2.0 ** -8, 2.0 ** -11  # half a step


def attend(q, k, v, r, p):
    """q [n, d] scaled queries, k and v [m, d], all in 64 bits -> output [n, d] and its bound."""
    x = q @ k.T
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    D = r * (np.abs(q) @ np.abs(k).T)
    o, size = w @ v, w @ np.abs(v)
    logits = (w * D) @ np.abs(v) + size * (w * D).sum(-1, keepdims=True)
    return o, BF16 * np.abs(o) + 1.1 * (logits + p * size) + 2.0 ** -12 * size


def assert_bounded(got, ref, bound, what):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    over = np.abs(got - ref) / bound
    assert over.max() <= 1, f"{what}: error up to {over.max():.3g} times its bound, at |o| {np.abs(ref).flat[over.argmax()]:.3g}"
