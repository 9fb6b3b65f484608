"""GPU tests of the base stream with attention sinks and of its gradient against plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
from synthetic import bf16_to_f32, normal_bf16, scale_offset
from tests import sink_util
from tests.attend_util import assert_bounded
from tests.gpu_util import bf, bits, dev, f32, val

pytestmark = pytest.mark.gpu


def f64(x):
    return bf16_to_f32(x).astype(np.float64)


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=dev())


class Stream:
    def __init__(self, B, T, Hq, Hkv, d, window, sinks, seed=1):
        self.x, self.dO = (normal_bf16(seed, n, (B, T, Hq, d)) for n in ("q_raw", "dO"))
        self.k, self.v = (normal_bf16(seed, n, (B, T, Hkv, d)) for n in ("k", "v"))
        self.alpha, self.beta = scale_offset(seed, Hq, d)
        self.window, self.sinks = window, sinks

    def reference(self):
        return sink_util.sink_fwd(f64(self.x), f64(self.k), f64(self.v), self.alpha.astype(np.float64),
                                  self.beta.astype(np.float64), self.window, self.sinks)

    def gradient(self, **kw):
        return sink_util.sink_bwd(f64(self.x), f64(self.k), f64(self.v), self.alpha.astype(np.float64),
                                  self.beta.astype(np.float64), f64(self.dO), self.window, self.sinks, **kw)

    def run(self, **kw):
        return orth.swa_sink_fwd(bf(self.x), bf(self.k), bf(self.v), f32(self.alpha), f32(self.beta), self.sinks,
                                 window=self.window, **kw)

    def run_bwd(self, **kw):
        o, lse = self.run(lse=True)
        return orth.swa_sink_bwd(bf(self.x), bf(self.k), bf(self.v), f32(self.alpha), f32(self.beta), o, bf(self.dO), lse,
                                 self.sinks, window=self.window, **kw)


CASES = [
    (1, 1, 2, 1, 64, 1, 1),          # one row
    (1, 2, 2, 1, 64, 1, 1),          # the first row that sees a sink behind its window
    (2, 33, 4, 4, 64, 5, 32),        # more sinks than most rows reach
    (1, 129, 4, 1, 128, 128, 4),     # one row behind the window
    (1, 130, 4, 1, 128, 128, 4),
    (2, 513, 2, 1, 64, 128, 4),      # G = 2
    (1, 700, 8, 2, 128, 128, 4),     # G = 4
    (3, 401, 8, 2, 64, 77, 5),
    (2, 300, 8, 1, 128, 33, 16),     # G = 8
    (1, 555, 16, 1, 128, 128, 17),   # G = 16
    (1, 260, 16, 1, 64, 1, 32),
    (2, 290, 3, 3, 128, 100, 31),    # G = 1
    (1, 900, 4, 2, 128, 300, 8),     # windows beyond tensor memory
    (1, 800, 4, 1, 64, 500, 32),
    (5, 200, 8, 2, 128, 64, 2),      # many short sequences: a CTA goes through several
    (9, 140, 16, 4, 64, 31, 3),
    (40, 161, 8, 2, 128, 128, 1),    # more streams than the grid has turns for at once
]


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", CASES)
def test_forward_matches(B, T, Hq, Hkv, d, window, sinks):
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T)
    ref, bound, ref_lse = s.reference()
    err = error_word()
    o = s.run(dev_err=err)
    assert_bounded(val(o), ref, bound, "o")
    o2, lse = s.run(lse=True, dev_err=err)
    np.testing.assert_array_equal(bits(o2), bits(o))
    # a logit is off by 2^-11 |q|.|k| (a few units in the sum of its products): 1e-2 as for the plain stream
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= 1e-2
    assert int(err.item()) == 0


@pytest.mark.parametrize("window", [1, 128, 300])
def test_no_sinks_and_wide_windows_are_the_plain_stream(window):
    s = Stream(2, 300, 8, 2, 128, window, 0, seed=3)
    plain = orth.swa_fwd(bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), window=window)
    np.testing.assert_array_equal(bits(s.run()), bits(plain))
    s.window, s.sinks = 300, 32
    plain = orth.swa_fwd(bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), window=300)
    np.testing.assert_array_equal(bits(s.run()), bits(plain))


@pytest.mark.parametrize("Hq,Hkv,d,window", [(8, 2, 128, 128), (8, 2, 64, 128), (2, 2, 128, 128), (8, 2, 128, 400)])
def test_row_ranges(Hq, Hkv, d, window):
    """Chunks give the bits of the whole, and no other row is written."""
    T = 900
    s = Stream(2, T, Hq, Hkv, d, window, 4, seed=4)
    whole, whole_lse = s.run(lse=True)
    out = torch.full((2, T, Hq, d), 7.0, dtype=torch.bfloat16, device=dev())
    lse = torch.full((2, T, Hq), 7.0, device=dev())
    s.run(out=out, lse=lse, row_begin=256, row_end=512)
    np.testing.assert_array_equal(bits(out[:, 256:512]), bits(whole[:, 256:512]))
    assert torch.equal(lse[:, 256:512], whole_lse[:, 256:512])
    for y in (out, lse):
        assert (y[:, :256] == 7).all() and (y[:, 512:] == 7).all()
    s.run(out=out, lse=lse, row_begin=0, row_end=256)
    s.run(out=out, lse=lse, row_begin=512)
    np.testing.assert_array_equal(bits(out), bits(whole))
    assert torch.equal(lse, whole_lse)


def test_strides_streams_and_graphs():
    """Batch strides above dense, appended query rows, another stream, a replayed graph: the same bits."""
    B, T, Hq, Hkv, d = 3, 333, 8, 2, 128
    s = Stream(B, T, Hq, Hkv, d, 128, 4, seed=5)
    ref = bits(s.run())

    def wide(x, n):
        y = torch.full((B, x.shape[1] + n) + x.shape[2:], float("nan"), dtype=torch.bfloat16, device=dev())
        y[:, :x.shape[1]] = bf(x)
        return y
    q, k, v = wide(s.x, 3), wide(s.k, 5)[:, :T], wide(s.v, 5)[:, :T]
    out = torch.full((B, T + 2, Hq, d), 3.0, dtype=torch.bfloat16, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = f32(s.alpha), f32(s.beta)
    with torch.cuda.stream(side):
        orth.swa_sink_fwd(q, k, v, a, b, 4, out=out[:, :T])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(out[:, :T]), ref)
    assert (out[:, T:] == 3.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orth.swa_sink_fwd(q, k, v, a, b, 4, out=out[:, :T])
    for _ in range(2):
        out.zero_()
        graph.replay()
        np.testing.assert_array_equal(bits(out[:, :T]), ref)


@pytest.mark.parametrize("Hq,Hkv,window", [(8, 2, 128), (2, 2, 128), (8, 2, 500)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_rows_behind_the_sinks_do_not_reach_far(Hq, Hkv, window, value):
    """Row 20 shares its key block with the sinks but is none: it does not reach rows more than window + 256 away."""
    s = Stream(1, 1000, Hq, Hkv, 128, window, 4, seed=6)
    clean = s.run()
    v = bf(s.v)
    v[:, 20] = value
    got = orth.swa_sink_fwd(bf(s.x), bf(s.k), v, f32(s.alpha), f32(s.beta), 4, window=window)
    far = 20 + window + 256
    np.testing.assert_array_equal(bits(got[:, far:]), bits(clean[:, far:]))
    assert not torch.isfinite(got[:, 20].float()).any()


@pytest.mark.parametrize("Hq,Hkv,window", [(8, 2, 128), (2, 2, 128), (8, 2, 500)])
def test_keys_beyond_fp16(Hq, Hkv, window):
    """Sinks (and keys of the window) of 2^17 times their size, the queries as much smaller."""
    s = Stream(1, 700, Hq, Hkv, 128, window, 5, seed=7)
    for j in (0, 3, 300):
        s.k[0, j] += 17 << 7  # bf16 exponent: times 2^17
    s.x -= 14 << 7
    s.x[(s.x & 0x7F80) == 0x7F80] = 0
    s.x[(s.x & 0x7F80) > (s.x & 0x7F80).dtype.type(140 << 7)] = 0
    s.beta[:] = 0
    ref, bound, _ = s.reference()
    err = error_word()
    got = s.run(dev_err=err)
    assert_bounded(val(got), ref, bound, "o")
    assert int(err.item()) == 0


def grad_parity(got, ref, what):
    """The bar of this repository's gradients: rounded operands (2^-9 each, random) move a tensor by a small multiple
    of 2^-9 of its norm, and no element by more than 3 % of the largest."""
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), what
    assert np.linalg.norm(got - ref) <= 1e-2 * np.linalg.norm(ref) + 1e-4, what
    assert np.abs(got - ref).max() <= 3e-2 * np.abs(ref).max() + 1e-4, what


NAMES = ("dq", "dk", "dv", "dalpha", "dbeta")


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", CASES + [(2, 64, 8, 2, 64, 128, 4), (3, 5, 16, 1, 128, 77, 1),
                                                              (1, 200, 4, 2, 64, 200, 0), (2, 100, 8, 1, 128, 33, 31)])
def test_log_sum_exp_of_few_keys(B, T, Hq, Hkv, d, window, sinks):
    """Rows that see at most 64 keys.  q enters as a bf16 part and a bf16 residual: 2^-9 2^-9 of each value off at most,
    so a logit, and with it the sum's logarithm, by 2^-18 of the sum of its products' sizes; fp32 sums, exponents and
    the logarithm add a few 2^-22 of it and of the result (at least 1 counted)."""
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + 3)
    _, lse = s.run(lse=True)
    ref = s.reference()[2]
    q = np.abs(f64(s.x) * s.alpha.astype(np.float64) + s.beta.astype(np.float64)) / np.sqrt(d)
    size = np.stack([q[:, :, h] @ np.abs(f64(s.k)[:, :, h * Hkv // Hq]).max(1)[..., None] for h in range(Hq)], 2)[..., 0]
    t = np.arange(T)
    few = np.minimum(t + 1, window) + np.minimum(sinks, np.maximum(0, t + 1 - window)) <= 64
    if window + sinks > 64:
        few &= t < 64
    off = np.abs(lse.cpu().numpy() - ref)[:, few]
    assert (off <= (2.0 ** -18 + 2.0 ** -20) * size[:, few] + 2.0 ** -20 * np.maximum(1, np.abs(ref[:, few]))).all()


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", CASES)
def test_gradient_matches(B, T, Hq, Hkv, d, window, sinks):
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + 1)
    err = error_word()
    got = s.run_bwd(dev_err=err)
    for g, ref, what in zip(got, s.gradient(), NAMES):
        grad_parity(g, ref, what)
    assert int(err.item()) == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", CASES)
def test_gradient_to_its_type(B, T, Hq, Hkv, d, window, sinks):
    """Given the same o and log-sum-exp.  q, dS and P are off by 2^-17 of their size at most (a bf16 residual of a bf16
    rounding: half a step of each, 2^-9 2^-8), which reaches a logit as 2^-17 |q|.|k| scale, some 2^-16 for these
    inputs, random in sign: three roundings of dk come to no more than 2^-15 of a tensor's norm, and no element is off
    by more than 2^-12 of the largest."""
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + 2)
    o, lse = s.run(lse=True)
    got = orth.swa_sink_bwd(bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), o, bf(s.dO), lse, sinks, window=window)
    want = s.gradient(o=val(o), lse=lse.cpu().numpy().astype(np.float64))
    for g, ref, what in zip(got, want, NAMES):
        g = g.cpu().numpy().astype(np.float64)
        assert np.linalg.norm(g - ref) <= 2.0 ** -15 * np.linalg.norm(ref) + 1e-5, what
        assert np.abs(g - ref).max() <= 2.0 ** -12 * np.abs(ref).max() + 1e-5, what


def test_sinks_own_gradient():
    """The sinks' rows of dk and dv alone, which many rows add to: held to the bar by themselves."""
    s = Stream(2, 1500, 8, 2, 128, 64, 20, seed=9)
    got, ref = s.run_bwd(), s.gradient()
    for i in (1, 2):
        grad_parity(got[i][:, :20], ref[i][:, :20], NAMES[i])


@pytest.mark.parametrize("Hq,Hkv,window", [(8, 2, 128), (16, 1, 128), (2, 2, 128), (4, 2, 300)])
def test_gradient_with_zeros_in_alpha(Hq, Hkv, window):
    s = Stream(1, 500, Hq, Hkv, 64, window, 4, seed=10)
    s.alpha[:, ::3] = 0
    for g, ref, what in zip(s.run_bwd(), s.gradient(), NAMES):
        grad_parity(g, ref, what)


def test_gradient_workspace_and_no_sinks():
    """The workspace may hold anything; without sinks it is the plain stream's gradient."""
    s = Stream(2, 400, 8, 2, 128, 128, 4, seed=11)
    n = orth.swa_sink_bwd_workspace_size(2, 400, 8, 2, 128)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev())
    for g, ref, what in zip(s.run_bwd(workspace=ws), s.gradient(), NAMES):
        grad_parity(g, ref, what)
    s.sinks = 0
    o, lse = s.run(lse=True)
    plain = orth.swa_bwd(bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), o, bf(s.dO), lse=lse)
    for g, ref, what in zip(s.run_bwd(workspace=ws), plain, NAMES):
        grad_parity(g, ref.cpu().numpy().astype(np.float64), what)


def test_gradient_in_a_graph():
    s = Stream(1, 300, 8, 2, 128, 128, 4, seed=12)
    o, lse = s.run(lse=True)
    args = [bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), o, bf(s.dO), lse, 4]
    ws = torch.empty(orth.swa_sink_bwd_workspace_size(1, 300, 8, 2, 128), dtype=torch.uint8, device=dev())
    eager = orth.swa_sink_bwd(*args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orth.swa_sink_bwd(*args, workspace=ws)
    for _ in range(2):
        for g in got:
            g.zero_()
        graph.replay()
        for i, (g, e) in enumerate(zip(got, eager)):
            if i < 3:  # dalpha, dbeta are summed with atomics
                assert torch.equal(g, e), NAMES[i]
            else:
                grad_parity(g, e.cpu().numpy().astype(np.float64), NAMES[i])


@pytest.mark.parametrize("sinks", [4, 0])
def test_gradients_one_after_the_other(sinks):
    """Calls of different sizes that share a workspace, whose last kernels run side by side: what follows a call in its
    stream (here the workspace is overwritten, the outputs are copied) finds it complete."""
    sizes = [(4, 1500, 8, 2), (1, 140, 4, 4), (2, 4000, 16, 2)]
    streams = [Stream(B, T, Hq, Hkv, 128, 128, sinks, seed=T) for B, T, Hq, Hkv in sizes]
    n = max(orth.swa_sink_bwd_workspace_size(B, T, Hq, Hkv, 128) for B, T, Hq, Hkv in sizes)
    calls = []
    for s in streams:
        o, lse = s.run(lse=True)
        calls.append((bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), o, bf(s.dO), lse, sinks))
    alone = []
    for c in calls:
        alone.append(orth.swa_sink_bwd(*c))
        torch.cuda.synchronize()
    ws = torch.empty(n, dtype=torch.uint8, device=dev())
    got = []
    for c in calls + calls[::-1]:
        y = orth.swa_sink_bwd(*c, workspace=ws)
        ws.fill_(0xFF)
        got.append([t.clone() for t in y])
        for t in y:
            t.fill_(float("nan"))
    for y, ref in zip(got, alone + alone[::-1]):
        for i in range(5):
            if i < 3:  # dalpha, dbeta are summed with atomics
                assert torch.equal(y[i], ref[i]), NAMES[i]
            else:
                grad_parity(y[i], ref[i].cpu().numpy().astype(np.float64), NAMES[i])


def test_offsets_beyond_32_bits():
    """Five sequences of 131072 rows of 32 heads: the last one's values lie beyond 2^31.  It comes out as alone (the
    sinks' dk and dv are sums of another number of parts, 32 or 38 runs of tokens: a part's sum is truncated at up to
    5 products of 64 steps, 320 2^-23 < 2^-14 of its size, random signs make that size a sixth of the whole's, and
    38 such errors of one sign come to 38/6 2^-14 < 2^-11 of the largest)."""
    B, T, Hq, Hkv, d = 5, 131072, 32, 8, 128
    gen = torch.Generator(device=dev()).manual_seed(3)
    x, dO = (torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    k, v = (torch.empty((B, T, Hkv, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    for t in (x, dO, k, v):
        for b in range(B):
            t[b].copy_(torch.randn(t.shape[1:], generator=gen, device=dev()))
    alpha, beta = (f32(a) for a in scale_offset(3, Hq, d))
    o, lse = orth.swa_sink_fwd(x, k, v, alpha, beta, 4, lse=True)
    y = orth.swa_sink_bwd(x, k, v, alpha, beta, o, dO, lse, 4)
    one = [t[4:].contiguous() for t in (x, k, v, dO)]
    o1, lse1 = orth.swa_sink_fwd(one[0], one[1], one[2], alpha, beta, 4, lse=True)
    assert torch.equal(o[4:], o1) and torch.equal(lse[4:], lse1)
    y1 = orth.swa_sink_bwd(one[0], one[1], one[2], alpha, beta, o1, one[3], lse1, 4)
    assert torch.equal(y[0][4:], y1[0])
    for i in (1, 2):
        assert torch.equal(y[i][4:, 4:], y1[i][:, 4:]), NAMES[i]
        far = (y[i][4:, :4] - y1[i][:, :4]).abs().max()
        assert far <= 2.0 ** -11 * y1[i][:, :4].abs().max(), NAMES[i]


@pytest.mark.parametrize("Hq,Hkv,window", [(8, 2, 9), (16, 1, 40), (2, 2, 128)])
def test_log_sum_exp_of_row_ranges(Hq, Hkv, window):
    """A range gives a row the bits that the whole stream gives it, and writes no other."""
    s = Stream(2, 300, Hq, Hkv, 128, window, 3, seed=15)
    _, whole = s.run(lse=True)
    for begin, end in ((0, 128), (128, 300), (128, 256), (256, 300), (256, 256)):
        lse = torch.full((2, 300, Hq), 7.0, device=dev())
        s.run(lse=lse, row_begin=begin, row_end=end)
        assert torch.equal(lse[:, begin:end], whole[:, begin:end])
        assert (lse[:, :begin] == 7.0).all() and (lse[:, end:] == 7.0).all()
