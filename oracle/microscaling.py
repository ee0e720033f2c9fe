"""Definitions in 64 bits of the microscaled formats and of the operators over them -- TEST INFRASTRUCTURE.

Blocks of 32 values with a shared power of two, quantized by looking the nearest element up in the list of the
format's magnitudes; the linear layer over MXFP4 weights.  No code is shared with the GPU library."""
from __future__ import annotations

import numpy as np

from oracle import serving

# magnitudes in the order of their codes, and floor(log2) of the largest
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
MAGNITUDES = {"mxfp4": E2M1, "mxfp8": E4M3}
TOP_EXPONENT = {"mxfp4": 2, "mxfp8": 8}


def nearest(a, magnitudes):
    """Index of the nearest magnitude of a >= 0, ties to the even index, the largest beyond the end."""
    half = (magnitudes[1:] + magnitudes[:-1]) / 2
    low, high = np.searchsorted(half, a, side="left"), np.searchsorted(half, a, side="right")
    return np.where(low % 2 == 0, low, high)


def quantize(x, form):
    """(codes, scales) uint8 of float64 values [..., n] that a type of at most 8 bits of exponent holds."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - TOP_EXPONENT[form], -127)
    e = np.maximum(e, -127)
    index = nearest(np.ldexp(np.abs(b), -e[..., None]), MAGNITUDES[form])
    sign = np.signbit(b) & ~bad[..., None]
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    if form == "mxfp8":
        return (index | (sign << 7)).astype(np.uint8).reshape(x.shape), scales
    nibbles = (index | (sign << 3)).reshape(x.shape)
    return (nibbles[..., ::2] | (nibbles[..., 1::2] << 4)).astype(np.uint8), scales


def dequantize(codes, scales, form):
    """float64 values [..., n] of codes and scales."""
    codes = np.asarray(codes)
    if form == "mxfp4":
        c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
        v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    else:
        v = np.where(codes & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 127]
    s = np.where(np.asarray(scales) == 255, np.nan, np.ldexp(1.0, np.asarray(scales).astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def _sum_error(x, W):
    """(z, bound): z = x W^T and how far sums of its products in fp32 on the matrix cores may be off.

    Products of elements and their scales are exact.  An instruction adds 64 or 128 of them to a sum; each of its
    additions, in whatever order, is within 2^-23 (they need not round to nearest) of what it can reach: |S| + A, S the sum
    in front of the instruction, A its sum of |x| |W|.  65 additions an instruction of 64 (an instruction of 128 counts as
    two), in one of the kernels' orders: a running sum over all instructions, or up to 16 of them over every 16th or so,
    joined by as many additions more.  |S| is bounded by the running sum of |x W| over a block of 64 either way, taken
    here as the sum of A so far: an upper bound of both."""
    z = x @ W.T
    reach, bound = np.zeros_like(z), np.zeros_like(z)
    for k in range(0, x.shape[1], 64):
        reach += np.abs(x[:, k:k + 64]) @ np.abs(W[:, k:k + 64]).T
        bound += reach
    return z, 2.0 ** -23 * (65 * bound + 16 * reach)


def mxfp4_linear(x, W, bias=None, residual=None, act="none", gated=False, out_type="bf16"):
    """(y, tol) of the layer's epilogue behind x W^T: x float64 [M, in] and W [cols, in] as they are after quantization;
    tol as of oracle.serving.w4a16_linear."""
    z, ez = _sum_error(x, W)
    if bias is not None:
        z = z + bias
        ez = ez + 2.0 ** -23 * np.abs(z)
    n = z.shape[1] // 2 if gated else z.shape[1]
    y = serving.activation(z[:, :n], act)
    e = serving._slope(z[:, :n], ez[:, :n], act) * ez[:, :n] + serving._activation_error(z[:, :n], y, act)
    if gated:
        up, eu = z[:, n:], ez[:, n:]
        e = e * np.abs(up) + (np.abs(y) + e) * eu + 2.0 ** -24 * np.abs(y * up)
        y = y * up
    if residual is not None:
        y = y + residual
        e = e + 2.0 ** -24 * np.abs(y)
    return y, e + serving.UNIT[out_type] * (np.abs(y) + e) + serving.TINY[out_type]
