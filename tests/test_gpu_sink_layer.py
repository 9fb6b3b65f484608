"""GPU test of a layer's training step with sinks: both streams forward with their log-sum-exp, then the base stream's
gradient and the copies' added into its dk and dv."""
import numpy as np
import pytest
import torch

import long_context_attention_orthros_gb300 as orth
import oracle
from tests.gpu_util import bf, f32, i32
from tests.test_gpu_sinks import NAMES, Stream, error_word, grad_parity
from tests.test_gpu_xattn_bwd import _copies

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,T_out,Hq,Hkv,d,window,sinks,positions", [
    (2, 400, 48, 16, 4, 128, 128, 4, "tail_shuffled"),
    (1, 300, 20, 8, 2, 64, 33, 16, "random"),
    (2, 700, 1, 32, 8, 128, 128, 4, "tail_shuffled"),
    (1, 130, 130, 8, 1, 64, 64, 1, "every"),
    (1, 260, 9, 3, 3, 128, 200, 32, "random"),
])
def test_training_step(B, T, T_out, Hq, Hkv, d, window, sinks, positions):
    """Held to the bar of this repository's gradients, which is that of the copies' rounded operands; the step is run
    twice on one stream without a wait between the calls, and both gradients' own parts are as alone."""
    s = Stream(B, T, Hq, Hkv, d, window, sinks, seed=T + T_out)
    qc, pos, dOc, ac, bc = _copies(T + T_out, B, T, T_out, Hq, d, positions)
    q, k, v, a, b, dO = bf(s.x), bf(s.k), bf(s.v), f32(s.alpha), f32(s.beta), bf(s.dO)
    qcg, pg, dOcg, acg, bcg = bf(qc), i32(pos), bf(dOc), f32(ac), f32(bc)
    err = error_word()
    for _ in range(2):
        o, lse = orth.swa_sink_fwd(q, k, v, a, b, sinks, window=window, lse=True, dev_err=err)
        oc, lsec = orth.xattn_fwd(qcg, pg, k, v, acg, bcg, lse=True, dev_err=err)
        dq, dk, dv, da, db = orth.swa_sink_bwd(q, k, v, a, b, o, dO, lse, sinks, window=window, dev_err=err)
        dqc, dk2, dv2, dac, dbc = orth.xattn_bwd(qcg, pg, k, v, acg, bcg, oc, dOcg, dk=dk, dv=dv, lse=lsec, dev_err=err)
        assert dk2 is dk and dv2 is dv
        rc = oracle.xattn_bwd(qc, pos, s.k, s.v, ac, bc, dOc, d ** -0.5)
        rb = s.gradient()
        for g, ref, what in zip((dq, dk, dv, da, db), (rb[0], rb[1] + rc[1], rb[2] + rc[2], rb[3], rb[4]), NAMES):
            grad_parity(g, ref, what)
        for g, ref, what in zip((dqc, dac, dbc), (rc[0], rc[3], rc[4]), ("dqc", "dalpha_c", "dbeta_c")):
            grad_parity(g, ref, what)
    assert int(err.item()) == 0
