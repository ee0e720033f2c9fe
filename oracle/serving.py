"""Definitions in 64 bits of the operators that run a packed checkpoint -- TEST INFRASTRUCTURE.

The linear layer over GPTQ-v1 tensors with its epilogue, the paged cache's block tables and slot
maps, and attention over that cache, in numpy with a loop over everything that has one; with each
the sums that the tests' error bounds are made of.  No code is shared with the GPU library."""
from __future__ import annotations

import math

import numpy as np

import oracle

# unit roundoff 2^-p (p significant bits: 8, 11, 24) and half the smallest subnormal of the types
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _tanh_argument(z):
    return 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)


def activation(z, act):
    z = np.asarray(z, np.float64)
    if act == "none":
        return z
    if act == "relu":
        return np.maximum(z, 0.0)
    with np.errstate(over="ignore"):
        if act == "silu":
            return z / (1.0 + np.exp(-z))
        if act == "gelu":
            return 0.5 * z * _erfc(-z / math.sqrt(2.0))
        if act == "gelu_tanh":
            return z / (1.0 + np.exp(-_tanh_argument(z)))  # (1 + tanh(u / 2)) / 2, without its cancellation
    raise ValueError(act)


def _slope(z, ez, act):
    """Bound of |act'| over [z - ez, z + ez].  Everywhere at most 1.13.  Left of 0 it falls with the value: for
    g(z) = z S(z), S the sigmoid or the normal distribution function, |g'| <= S + |z| S', where S' is at most S u'
    (sigmoid of u) or, of the distribution, (|z| + 1 / |z|) S; all grow with z or |z|, taken at their ends."""
    if act in ("none", "relu"):
        return np.ones_like(z)
    hi, far = z + ez, np.abs(z) + ez
    with np.errstate(over="ignore"):
        if act == "silu":
            left = (1.0 + far) / (1.0 + np.exp(-hi))
        elif act == "gelu":
            left = (far * far + 2.0) * 0.5 * _erfc(-hi / math.sqrt(2.0))
        else:
            left = (1.0 + far * (1.6 + 0.22 * far * far)) / (1.0 + np.exp(-_tanh_argument(hi)))
    return np.where(hi < 0, np.minimum(left, 1.13), 1.13)


def _activation_error(z, y, act):
    """Bound of the fp32 evaluation's own error at z, y = act(z): each rounding 2^-24, the hardware's exponential
    2^-23, the tail of the normal distribution 16 units (2^-19).  A relative error of an argument moves the exponential or erfc by that times the
    argument, left of 0 as much in relative terms of the value:
      silu       z / (1 + e^-z): two roundings of the exponent, then 8 at most;
      gelu       z erfc(-z / sqrt 2) / 2: two roundings of the argument, whose factor is at most z^2 + 1;
      gelu_tanh  z / (1 + e^-u): eight roundings of u, two of the exponent, then 9;
    and what lies below the smallest normal numbers (e^-88 z and less) may be 0."""
    if act in ("none", "relu"):
        return np.zeros_like(z)
    left = np.maximum(-z, 0.0)
    if act == "silu":
        rel = 2.0 ** -24 * (2.0 * left + 8.0)
    elif act == "gelu":
        rel = 2.0 ** -19 + 2.0 ** -23 * (left * left + 1.0)
    else:
        rel = 2.0 ** -24 * (10.0 * np.maximum(-_tanh_argument(z), 0.0) + 9.0)
    return rel * np.abs(y) + 2.0 ** -120


def _sum_error(x, W):
    """(z, bound): z = x W^T and how far fp32 sums of its exact products may be off.

    The matrix cores add blocks of products to a sum: 32 additions a block of 32 and the block's own two roundings,
    each within 2^-23 (they need not round to nearest) of what the sum or the block can reach, |S| + A with S the sum in
    front of the block and A the block's sum of |x| |W|.  What is rounded is S itself, in one of two orders: group by
    group, each group's sum scaled and added (an fma each, and a join of up to 8), or one running sum over all
    groups, held in units of the group's scale: two roundings more a group for the change of units and two at
    the end.  The bound is the larger of the two, with 2^-10 of itself for the sums' own deviations."""
    total, own = (np.zeros((x.shape[0], W.shape[0])) for _ in range(2))  # sums over all groups, over this one
    blocks = np.zeros_like(total)                                        # sum of A
    running, within, turns, groups = (np.zeros_like(total) for _ in range(4))
    for k in range(0, x.shape[1], 32):
        if k % 128 == 0:
            turns += np.abs(total)
            groups += np.abs(own)
            own[:] = 0
        running += np.abs(total)
        within += np.abs(own)
        blocks += np.abs(x[:, k:k + 32]) @ np.abs(W[:, k:k + 32]).T
        part = x[:, k:k + 32] @ W[:, k:k + 32].T
        total += part
        own += part
    groups += np.abs(own)
    G = x.shape[1] // 128
    chain = 34 * 2.0 ** -23 * (running + blocks) + 2.0 ** -23 * (turns + np.abs(total))
    apart = 34 * 2.0 ** -23 * (within + blocks) + 2.0 ** -24 * (G + 8) * groups
    return total, (1 + 2.0 ** -10) * np.maximum(chain, apart)


def w4a16_linear(x, qweight, scales, bias=None, residual=None, act="none", gated=False, out_type="bf16"):
    """(y, tol): x float64 [M, in] holding the 16-bit values, qweight int32 [in/8, cols], scales
    uint16 binary16 bits [in/128, cols].

    tol: _sum_error for z and a rounding for the bias; the activation has _slope and its own _activation_error;
    then the product with the up half, the residual's sum and the rounding of y."""
    x = np.asarray(x, np.float64)
    codes, sbits = oracle.unpack_gptq_v1(qweight, scales)      # [cols, in], [cols, in/128]
    s = np.asarray(sbits).view(np.float16).astype(np.float64)
    W = codes.astype(np.float64) * np.repeat(s, 128, axis=1)
    z, ez = _sum_error(x, W)
    if bias is not None:
        z = z + bias
        ez = ez + 2.0 ** -23 * np.abs(z)
    n = z.shape[1] // 2 if gated else z.shape[1]
    y = activation(z[:, :n], act)
    e = _slope(z[:, :n], ez[:, :n], act) * ez[:, :n] + _activation_error(z[:, :n], y, act)
    if gated:
        up, eu = z[:, n:], ez[:, n:]
        e = e * np.abs(up) + (np.abs(y) + e) * eu + 2.0 ** -24 * np.abs(y * up)
        y = y * up
    if residual is not None:
        y = y + residual
        e = e + 2.0 ** -24 * np.abs(y)
    return y, e + UNIT[out_type] * (np.abs(y) + e) + TINY[out_type]


def block_map(ctx_len, new_len, free_pages, n_free, block_table, page_size, max_tokens):
    """The dict of cq.kv_block_map, with the updated block_table, request by request."""
    R, most = block_table.shape
    table = np.array(block_table, np.int64)
    n_free = min(max(int(n_free), 0), len(free_pages))
    left, tokens, stopped = n_free, 0, False
    cu, kv, status = [0], [], []
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    for r in range(R):
        ctx, new = int(ctx_len[r]), int(new_len[r])
        if ctx < 0 or new < 0 or ctx + new > most * page_size:
            status.append(2)
            kv.append(max(ctx, 0))
            cu.append(tokens)
            continue
        have, want = -(-ctx // page_size), -(-(ctx + new) // page_size)
        if stopped or want - have > left or tokens + new > max_tokens:
            stopped = True
            status.append(1)
            kv.append(ctx)
            cu.append(tokens)
            continue
        for b in range(have, want):
            left -= 1
            table[r, b] = free_pages[left]
        for i in range(new):
            p = ctx + i
            page = table[r, p // page_size]
            slot = page * page_size + p % page_size
            slots[tokens + i] = slot if page >= 0 and slot < 1 << 31 else -1
            positions[tokens + i] = p
        tokens += new
        status.append(0)
        kv.append(ctx + new)
        cu.append(tokens)
    return {"cu_q": np.array(cu), "kv_len": np.array(kv, np.int64), "slots": slots, "positions": positions,
            "status": np.array(status, np.int64), "n_left": np.array([left]), "block_table": table}


def paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_len, scale, causal=True, window=0, type="bf16"):
    """(out, lse, tol, lse_tol): q [T, H, D], caches [pages, Hkv, page, D], float64 values of the 16-bit
    inputs; rows that no request owns are 0 / -inf.

    tol: a score is D products summed in fp32 and scaled, so |ds| <= (D + 2) 2^-24 scale sum |q||k|, plus
    2^-21 (1 + max |s|) for the exponential's argument (products with log2 e and the maximum's, each
    rounded) and value; numerator and denominator each carry that once; the weights are rounded to the 16-bit
    type (u relative, and half its smallest subnormal); n terms are summed in fp32 with at most as many
    rescalings; then the output's rounding."""
    T, H, D = q.shape
    n_pages, Hkv, page, _ = k_cache.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol, lse_tol = np.zeros((T, H, D)), np.zeros((T, H))
    u, tiny = UNIT[type], TINY[type]
    for r in range(len(kv_len)):
        n = int(cu_q[r + 1]) - int(cu_q[r])
        kv = min(int(kv_len[r]), block_table.shape[1] * page)
        for i in range(n):
            p = kv - n + i
            js = [j for j in range(kv) if (not causal or j <= p) and (not window or j > p - window)
                  and 0 <= block_table[r, j // page] < n_pages]
            if not js:
                continue
            pg, at = np.array([block_table[r, j // page] for j in js]), np.array([j % page for j in js])
            for h in range(H):
                kh = h // (H // Hkv)
                K, V = k_cache[pg, kh, at], v_cache[pg, kh, at]
                row = q[int(cu_q[r]) + i, h]
                s = scale * (K @ row)
                ds = (D + 2) * 2.0 ** -24 * abs(scale) * (np.abs(K) @ np.abs(row))
                m = s.max()
                w = np.exp(s - m)
                L = w.sum()
                w /= L
                ds = float(ds.max()) + 2.0 ** -21 * (1.0 + float(np.abs(s).max()))
                t = int(cu_q[r]) + i
                A = w @ np.abs(V)
                out[t, h] = w @ V
                lse[t, h] = m + np.log(L)
                rel = u + 4 * ds + (2 * len(js) + 64) * 2.0 ** -24
                e = rel * A + len(js) * tiny / L * np.abs(V).max(0)
                tol[t, h] = e + u * (np.abs(out[t, h]) + e) + tiny
                lse_tol[t, h] = 2 * ds + (len(js) + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[t, h])
    return out, lse, tol, lse_tol
