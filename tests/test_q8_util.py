"""The numpy definition of the 8-bit cache against torch's own e4m3 type and against closed forms (CPU)."""
import numpy as np
import pytest
import torch

from synthetic import bf16_bits, bf16_to_f32, normal_bf16
from tests.q8_util import LARGEST, code_values, e4m3_values, quantize, value_bits


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(e4m3_values().astype(np.float32), t)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_codes_are_the_nearest_and_exponents_the_smallest(code):
    x = normal_bf16(3, "k", (500, 64))
    x[0] = 0
    x[1, :] = 0x7F00  # 2^127
    x[2, :] = bf16_bits(np.array([448.0], np.float32))[0]
    x[3, :] = bf16_bits(np.array([450.0], np.float32))[0]
    x[4, :] = bf16_bits(np.array([127.0], np.float32))[0]
    x[5, :] = bf16_bits(np.array([127.5], np.float32))[0]
    c, e = quantize(x, code)
    v = bf16_to_f32(x).astype(np.float64)
    scaled = v * np.exp2(-e.astype(float))[:, None]
    assert e[0] == 0 and not c[0].any()
    assert np.abs(scaled).max() <= LARGEST[code]
    assert (np.abs(scaled[1:]).max(-1) * 2 > LARGEST[code]).all()  # e - 1 would not do
    if code == "e4m3":
        want = torch.from_numpy(scaled.astype(np.float32)).to(torch.float8_e4m3fn).float().numpy()
    else:
        want = torch.round(torch.from_numpy(scaled)).numpy()
    np.testing.assert_array_equal(code_values(c, code), want)
    # half a step at most: 2^-4 of the value for e4m3 (2^-10 below its normal range), half a code for int8
    back = bf16_to_f32(value_bits(c, e, code)).astype(np.float64) * np.exp2(-e.astype(float))[:, None]
    tol = np.maximum(np.abs(scaled) * 2.0 ** -4, 2.0 ** -10) if code == "e4m3" else 0.5
    assert (np.abs(back - scaled) <= tol).all()
