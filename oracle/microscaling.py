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


def _orders(n):
    """The orders in which n 128s of k may be summed: lists of runs, a sum each, that are added up one by one.

    All in one sum, or neighbours to one sum of 4 or 8, the same number to each but the last ones."""
    steps = list(range(n))
    orders = [[steps]]
    for w in (4, 8):
        each = -(-n // w)
        orders.append([steps[i:i + each] for i in range(0, n, each)])
    return orders


def _sum_error(x, W):
    """(z, bound): z = x W^T and how far sums of its products in fp32 on the matrix cores may be off.

    Products of elements with their scales are exact.  128 of them are added to a sum by one instruction, or by up to four
    (64 of k each, or an operand in two parts, whose zeros change nothing): 128 additions and, where an instruction rounds what
    it adds up before it adds it to the sum, four more.  Each is within 2^-23 (they need not round to nearest) of what the sum can
    reach on the way, |S| + A with S the sum in front of the 128 and A the sum of their |x| |W|.  The bound is the largest
    of those of the orders in which the 128s are summed."""
    n = x.shape[1] // 128
    z = x @ W.T
    parts = [x[:, 128 * k:128 * k + 128] @ W[:, 128 * k:128 * k + 128].T for k in range(n)]
    sizes = [np.abs(x[:, 128 * k:128 * k + 128]) @ np.abs(W[:, 128 * k:128 * k + 128]).T for k in range(n)]
    bound = np.zeros_like(z)
    for order in _orders(n):
        err, joined, size = np.zeros_like(z), np.zeros_like(z), np.zeros_like(z)
        for run in order:
            S = np.zeros_like(z)
            for k in run:
                err += 132 * 2.0 ** -23 * (np.abs(S) + sizes[k])
                S = S + parts[k]
            joined = joined + S
            size += np.abs(joined)
        bound = np.maximum(bound, err + 2.0 ** -24 * (size if len(order) > 1 else 0.0))
    return z, (1 + 2.0 ** -10) * bound


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
