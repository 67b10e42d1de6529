"""Cases for the tests of the 8-bit products and the layer of experts."""
import numpy as np
import torch

from oracle import experts as ref
from oracle.fp8_paged import e4m3_decode, e4m3_encode
from tests._fp8 import DEV, DTYPES, HALF_STEP, call_over_freed_blocks, dev, host

# A group's 128 products are exact in binary32; adding them up loses at most a
# step, 2^-23, of the group's magnitudes for each addition, 2^-16 in all; up to
# 128 groups are added with a rounding of 2^-24 each, 2^-17; a factor's two
# roundings are 2^-23. In all below 2^-15 of the sum of magnitudes.
SUMS = 2.0 ** -15


def codes(rng, shape, spread=2.0):
    """E4M3 codes and their fp32 scales by rows and groups of 128: rows of several sizes."""
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, (*shape[:-1], 1)))
    groups = -(-shape[-1] // 128)
    padded = np.zeros((*shape[:-1], groups * 128))
    padded[..., :shape[-1]] = x
    scales = (np.maximum(np.abs(padded).reshape(*shape[:-1], groups, 128).max(-1), 1e-4) / 448).astype(np.float32)
    return e4m3_encode(x / ref.spread(scales, shape[-1])), scales


def weights(rng, shape):
    """E4M3 codes [.., n, k] over most of their range and the fp32 scales of their blocks."""
    blocks = (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128))
    c = e4m3_encode(rng.standard_normal(shape) * 80)
    return c, (rng.uniform(0.5, 1.5, blocks) / (80 * np.sqrt(shape[-1]))).astype(np.float32)


def u8(x, pitch=None):
    """On the GPU, with `pitch` bytes from row to row (NaN codes between)."""
    t = torch.from_numpy(np.ascontiguousarray(x))
    if pitch is None:
        return t.to(DEV)
    wide = torch.full((*x.shape[:-1], pitch), 0x7F, dtype=torch.uint8)
    wide[..., :x.shape[-1]] = t
    return wide.to(DEV)[..., :x.shape[-1]]


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV)


def i64(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int64)).to(DEV)


def check_product(got, y, mass, dtype):
    d = np.abs(got.double().cpu().numpy() - y)
    assert np.all(d <= HALF_STEP[dtype] * np.abs(y) + 1.01 * SUMS * mass + 2.0 ** -25)


def check_gated(got, y, mass):
    """silu's exponential and quotient are within 2^-19 of their value, relative to it (arguments
    up to 64: the argument's rounding, 64 * 2^-24, and a few units in the last place)."""
    out, scales = got
    z, want, per = ref.gated(y, mass)
    off = 1.01 * SUMS * per + 2.0 ** -17 * np.abs(z) + 1e-30
    s = scales.double().cpu().numpy()
    most = off.reshape(len(z), -1, 128).max(2)
    assert np.all(np.abs(s - want) <= most / 448 + 2.0 ** -22 * want)
    full = np.repeat(s, 128, 1)
    value = e4m3_decode(host(out)) * full
    assert np.all(np.abs(value - z) <= 2.0 ** -4 * np.abs(z) + 2.0 ** -10 * full + 1.07 * off
                  + 448 * np.repeat(np.abs(s - want), 128, 1))


__all__ = ["DEV", "DTYPES", "HALF_STEP", "SUMS", "call_over_freed_blocks", "check_gated", "check_product", "codes", "dev",
           "e4m3_decode", "e4m3_encode", "f32", "host", "i64", "ref", "u8", "weights"]
