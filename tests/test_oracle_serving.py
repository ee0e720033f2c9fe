"""Pins of the oracle's serving operators (oracle/serving.py) on hand examples and on independent
forms, and planted mistakes that the pins would see."""
import math

import numpy as np
import pytest

import oracle
from oracle import serving


def _packed(codes, sv):
    out, inp = codes.shape
    return oracle.pack_gptq_v1(codes, sv.view(np.uint16), out, inp)


def test_linear_one_hot_rows_bias_and_residual():
    rng = np.random.default_rng(0)
    codes = rng.integers(-8, 8, (6, 256)).astype(np.int8)
    sv = rng.uniform(0.01, 0.1, (6, 2)).astype(np.float16)
    qw, sc = _packed(codes, sv)
    x = np.eye(256)[[0, 127, 128, 255]]
    b, r = np.arange(6.0), 10 * np.ones((4, 6))
    y, tol = serving.w4a16_linear(x, qw, sc, bias=b, residual=r)
    for i, k in enumerate((0, 127, 128, 255)):
        assert np.allclose(y[i], codes[:, k] * sv[:, k // 128].astype(np.float64) + b + 10, rtol=1e-15)
    assert np.all(tol > 0)


def test_activations_at_known_points():
    assert serving.activation(0.0, "silu") == 0 and serving.activation(0.0, "gelu") == 0
    assert math.isclose(serving.activation(1.0, "silu"), 1 / (1 + math.exp(-1)))
    assert math.isclose(serving.activation(1.0, "gelu"), 0.8413447460685429)
    assert math.isclose(serving.activation(1.0, "gelu_tanh"), 0.8411919906082768)
    assert serving.activation(-2.0, "relu") == 0 and serving.activation(2.0, "relu") == 2


def test_tanh_gelu_keeps_its_tail():
    """z (1 + tanh(u / 2)) / 2 = z / (1 + e^-u), whose value far below 0 is z e^u (1 + tanh itself cancels there)."""
    for z in (-2.0, -5.0, -7.0, -9.0):
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        want = z * math.exp(u) / (1 + math.exp(u))
        assert math.isclose(serving.activation(z, "gelu_tanh"), want, rel_tol=1e-13)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slope_bounds_the_differences(act):
    z = np.concatenate([np.linspace(-12, 6, 4001), np.linspace(-1e-3, 1e-3, 101)])
    for ez in (1e-9, 1e-4, 0.1, 2.0):
        s = serving._slope(z, np.full_like(z, ez), act)
        y = serving.activation(z, act)
        for dz in (-ez, -ez / 3, ez / 2, ez):
            assert np.all(np.abs(serving.activation(z + dz, act) - y) <= s * abs(dz) * (1 + 1e-6) + 1e-15 * np.abs(y))


@pytest.mark.parametrize("act,lost", [("gelu", lambda z: 0.5 * z * (1 + math.erf(z / math.sqrt(2)))),
                                      ("gelu_tanh", lambda z: 0.5 * z * (1 + math.tanh(0.7978845608 * (z + 0.044715 * z ** 3))))])
def test_planted_cancellation_exceeds_the_bound(act, lost):
    """1 + erf and 1 + tanh in binary32 leave the bound of a negative argument's value."""
    for z in (-4.0, -5.0, -6.0):
        want = serving.activation(z, act)
        bad = np.float32(0.5 * z) * (np.float32(1) + np.float32(lost(z) / (0.5 * z) - 1))
        assert abs(bad - want) > serving._activation_error(np.array(z), want, act)


def test_gated_takes_the_gate_first():
    codes = np.zeros((2, 128), np.int8)
    codes[0, 0], codes[1, 0] = 3, 5
    qw, sc = _packed(codes, np.ones((2, 1), np.float16))
    y, _ = serving.w4a16_linear(np.eye(128)[:1], qw, sc, act="silu", gated=True)
    assert math.isclose(y[0, 0], 3 / (1 + math.exp(-3)) * 5)


def test_block_map_by_hand():
    table = np.full((4, 3), -1)
    table[0, 0], table[1, :2] = 9, (8, 7)
    m = serving.block_map([3, 8, 0, 0], [2, 1, 0, 13], [1, 2, 3, 4], 4, table, 4, 16)
    assert list(m["status"]) == [0, 0, 0, 2]                       # 13 tokens exceed three pages of four
    assert list(m["cu_q"]) == [0, 2, 3, 3, 3]
    assert list(m["block_table"][0]) == [9, 4, -1] and list(m["block_table"][1]) == [8, 7, 3]
    assert list(m["slots"][:4]) == [9 * 4 + 3, 4 * 4, 3 * 4, -1]
    assert list(m["positions"][:4]) == [3, 4, 8, 0]
    assert m["n_left"][0] == 2 and list(m["kv_len"]) == [5, 9, 0, 0]


def test_block_map_refuses_from_the_first_that_does_not_fit():
    table = np.full((3, 4), -1)
    m = serving.block_map([0, 0, 0], [4, 9, 1], [5, 6, 7], 3, table, 4, 100)
    assert list(m["status"]) == [0, 1, 1] and m["n_left"][0] == 2 and list(m["cu_q"]) == [0, 4, 4, 4]


def _attention_inputs(rng, lens, H, Hkv, D, page):
    T = sum(n for n, _ in lens)
    pages = [-(-kv // page) for _, kv in lens]
    perm = rng.permutation(sum(pages) + 2)
    table = np.full((len(lens), max(pages + [1])), -1)
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = perm[at:at + p]
        at += p
    kc, vc = (rng.standard_normal((sum(pages) + 2, Hkv, page, D)) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
    return rng.standard_normal((T, H, D)), kc, vc, table, cu, np.array([kv for _, kv in lens])


def _dense(q, kc, vc, table, cu, kv_len, scale, causal, window):
    """The same by whole score matrices with an additive mask."""
    out = np.zeros_like(q)
    H, Hkv, page = q.shape[1], kc.shape[1], kc.shape[2]
    for r, kv in enumerate(kv_len):
        K = kc[table[r, :-(-kv // page)]].transpose(1, 0, 2, 3).reshape(Hkv, -1, q.shape[2])[:, :kv]
        V = vc[table[r, :-(-kv // page)]].transpose(1, 0, 2, 3).reshape(Hkv, -1, q.shape[2])[:, :kv]
        n = cu[r + 1] - cu[r]
        p, j = np.arange(kv - n, kv)[:, None], np.arange(kv)[None]
        bad = ((j > p) & causal) | ((j <= p - window) & (window > 0))
        for h in range(H):
            s = q[cu[r]:cu[r + 1], h] @ K[h * Hkv // H].T * scale
            s = np.where(bad, -np.inf, s)
            e = np.exp(s - s.max(1, keepdims=True))
            out[cu[r]:cu[r + 1], h] = e / e.sum(1, keepdims=True) @ V[h * Hkv // H]
    return out


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3)])
def test_attention_against_dense_matrices(causal, window):
    a = _attention_inputs(np.random.default_rng(1), [(3, 7), (1, 9), (5, 5)], 4, 2, 8, 4)
    out = serving.paged_attention(*a, 0.3, causal, window)[0]
    assert np.allclose(out, _dense(*a, 0.3, causal, window), atol=1e-13)


def test_attention_empty_rows():
    q, kc, vc, table, cu, kv = _attention_inputs(np.random.default_rng(2), [(4, 4), (2, 2)], 2, 1, 8, 4)
    out, lse, _, _ = serving.paged_attention(q, kc, vc, table, cu, np.array([2, 0]), 1.0)
    assert np.all(out[[0, 1, 4, 5]] == 0) and np.all(np.isneginf(lse[[0, 1, 4, 5]])) and np.all(lse[2:4] > -50)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0)])
def test_attention_lengths_past_the_table_are_those_of_the_table(causal, window):
    q, kc, vc, table, cu, kv = _attention_inputs(np.random.default_rng(4), [(4, 8), (2, 5)], 2, 1, 8, 4)
    assert table.shape[1] == 2
    want = serving.paged_attention(q, kc, vc, table, cu, kv, 1.0, causal, window)[0]
    got = serving.paged_attention(q, kc, vc, table, cu, np.array([8 + 100, kv[1]]), 1.0, causal, window)[0]
    assert np.array_equal(got, want)


def test_planted_mistakes_exceed_the_bounds():
    """A mask one key too wide, a head group off by one and a nibble order reversed all leave the bounds."""
    rng = np.random.default_rng(3)
    a = _attention_inputs(rng, [(6, 40), (1, 33)], 4, 2, 16, 8)
    out, _, tol, _ = serving.paged_attention(*a, 0.25, True, 0, "bf16")
    shifted = _dense(*a[:4], a[4], a[5], 0.25, True, 12)
    assert np.any(np.abs(shifted - out) > tol)
    swapped = serving.paged_attention(a[0], a[1][:, ::-1], a[2], *a[3:], 0.25)[0]
    assert np.any(np.abs(swapped - out) > tol)
    codes = rng.integers(-8, 8, (16, 256)).astype(np.int8)
    sv = rng.uniform(0.01, 0.05, (16, 2)).astype(np.float16)
    x = rng.standard_normal((3, 256))
    y, tol = serving.w4a16_linear(x, *_packed(codes, sv))
    rev = codes.reshape(16, 32, 8)[:, :, ::-1].reshape(16, 256)
    bad, _ = serving.w4a16_linear(x, *_packed(np.ascontiguousarray(rev), sv))
    assert np.mean(np.abs(bad - y) > tol) > 0.9


def _summed_in_fp32(x, codes, sv, chain, inner=np.float32, outer=np.float32):
    """x W^T as the kernels sum it: blocks of 16 exact products, one rounding a block (``inner``); groups of their own
    scaled in (``outer``), or one chain in units of the group's scale that is rescaled between groups."""
    x, codes = x.astype(np.float64), codes.astype(np.float64)
    s = sv.astype(np.float64)
    total, acc, last = np.zeros((len(x), len(codes)), outer), np.zeros((len(x), len(codes)), inner), None
    for g in range(s.shape[1]):
        if chain and g:
            ratio = (np.float32(s[:, g - 1]) / np.float32(s[:, g])).astype(np.float32)
            acc = (acc.astype(np.float64) * ratio).astype(inner)
        elif not chain:
            acc = np.zeros_like(acc)
        for k in range(128 * g, 128 * g + 128, 16):
            acc = (acc + x[:, k:k + 16] @ codes[:, k:k + 16].T).astype(inner)
        if not chain:
            total = (total + acc * s[:, g]).astype(outer)
    return (acc * s[:, -1]).astype(np.float32) if chain else total


@pytest.mark.parametrize("inp", [128, 1024, 4096])
def test_linear_bound_holds_for_fp32_sums_and_for_no_less(inp):
    """Both orders of the kernels' sums in fp32 stay within the bound; group sums or running sums held in binary16, a
    result rounded to binary16 in front of an fp32 store, and one code off by one leave it."""
    rng = np.random.default_rng(inp)
    codes = rng.integers(-8, 8, (48, inp)).astype(np.int8)
    sv = rng.uniform(1e-3, 2e-2, (48, inp // 128)).astype(np.float16)
    x = np.asarray(rng.standard_normal((64, inp)), np.float16).astype(np.float64)
    y, tol = serving.w4a16_linear(x, *_packed(codes, sv), out_type="f32")

    def outside(z):
        return np.mean(np.abs(z - y) > tol)

    for chain in (False, True):
        assert outside(_summed_in_fp32(x, codes, sv, chain)) == 0
        assert outside(_summed_in_fp32(x, codes, sv, chain, inner=np.float16)) > 0.2
    assert outside(_summed_in_fp32(x, codes, sv, False, outer=np.float16)) > 0.2
    assert outside(y.astype(np.float16).astype(np.float64)) > 0.01
    off = codes.copy()
    at = np.arange(48), rng.integers(0, inp, 48)
    off[at] += np.where(off[at] < 0, 1, -1).astype(np.int8)
    assert outside(_summed_in_fp32(x, off, sv, False)) > 0.7
