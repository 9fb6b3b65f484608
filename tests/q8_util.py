"""The 8-bit cache's definition in numpy, in 64 bits and apart from the kernels: codes, exponents and the
bf16 values they stand for."""
import numpy as np

from synthetic import bf16_to_f32

LARGEST = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The 256 e4m3 codes' values: 1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man / 8.0 * 2.0 ** -6, (1 + man / 8.0) * np.exp2(ex - 7.0))
    v = np.where(c & 0x7F == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def code_values(codes: np.ndarray, code: str) -> np.ndarray:
    return e4m3_values()[codes] if code == "e4m3" else codes.view(np.int8).astype(np.float64)


def quantize(bits: np.ndarray, code: str):
    """bf16 bits [..., d] -> (codes uint8 [..., d], exponents int8 [...]); every value finite."""
    x = bf16_to_f32(bits).astype(np.float64)
    amax = np.abs(x).max(-1)
    e = np.zeros(amax.shape, np.int64)
    nz = amax > 0
    e[nz] = np.ceil(np.log2(amax[nz] / LARGEST[code])).astype(np.int64)
    for _ in range(2):  # log2 is rounded: settle at the smallest e with amax 2^-e <= M
        e[nz & (amax * np.exp2(-e.astype(float)) > LARGEST[code])] += 1
        e[nz & (amax * np.exp2(-(e - 1).astype(float)) <= LARGEST[code])] -= 1
    e = np.clip(e, -126, 127)
    y = x * np.exp2(-e.astype(float))[..., None]
    if code == "int8":
        return np.rint(y).astype(np.int8).view(np.uint8), e.astype(np.int8)
    pos = e4m3_values()[:127]
    a = np.abs(y)
    lo = np.clip(np.searchsorted(pos, a, side="right") - 1, 0, 125)
    up = a - pos[lo] > pos[lo + 1] - a
    tie = a - pos[lo] == pos[lo + 1] - a
    c = lo + (up | (tie & (lo % 2 == 1)))
    return (c | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8), e.astype(np.int8)


def value_bits(codes: np.ndarray, e: np.ndarray, code: str) -> np.ndarray:
    """bf16 bits of the values code * 2^e (exact in bf16 for these exponents)."""
    v = code_values(codes, code) * np.exp2(e.astype(float))[..., None]
    f = v.astype(np.float32)
    u = f.view(np.uint32)
    fine = np.isfinite(v)
    assert np.array_equal(f[fine].astype(np.float64), v[fine]) and not np.any(u[fine] & 0xFFFF)
    return (u >> 16).astype(np.uint16)
