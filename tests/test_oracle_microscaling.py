"""The definitions of the microscaled formats, pinned by hand-worked blocks and by properties."""
import numpy as np
import pytest

from oracle import microscaling as mx


def _block(*values):
    return np.array(list(values) + [0.0] * (32 - len(values)))


def test_magnitudes():
    assert mx.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert len(mx.E4M3) == 127 and mx.E4M3[1] == 2.0 ** -9 and mx.E4M3[8] == 2.0 ** -6 and mx.E4M3[-1] == 448
    assert np.all(np.diff(mx.E4M3) > 0)


def test_a_block_by_hand():
    """Largest magnitude 7: scale 2^(2 - 2); 7 saturates at 6, ties go to the even code, the sign is bit 3."""
    codes, scales = mx.quantize(_block(7.0, -0.25, 0.75, 1.25, 1.75, 2.5, -3.5, 5.0), "mxfp4")
    assert scales.tolist() == [127]
    # 6, -0, 1, 1, 2, 2, -4, 4 -> codes 7, 8, 2, 2, 4, 4, 14, 6
    assert codes[:4].tolist() == [0x87, 0x22, 0x44, 0x6E] and not codes[4:].any()
    assert mx.dequantize(codes, scales, "mxfp4")[:8].tolist() == [6, 0, 1, 1, 2, 2, -4, 4]


def test_a_block_of_eight_bits_by_hand():
    """Largest magnitude 1: scale 2^-8; 1 is 256 units, code 0x78; 1.9999 would saturate at 448."""
    codes, scales = mx.quantize(_block(1.0, -1.96875, 2.0 ** -17, 2.0 ** -18, 3 * 2.0 ** -18), "mxfp8")
    assert scales.tolist() == [119]
    assert codes[:5].tolist() == [0x78, 0xFE, 0x01, 0x00, 0x02]


@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
def test_ends_of_the_scale(form):
    zero, tiny = mx.quantize(_block(0.0, -0.0), form), mx.quantize(_block(2.0 ** -133), form)
    assert zero[1].tolist() == [0] and tiny[1].tolist() == [0]
    assert mx.quantize(_block(2.0 ** 127 * 1.99), form)[1].tolist() == [254 - mx.TOP_EXPONENT[form]]
    for bad in (np.nan, np.inf, -np.inf):
        codes, scales = mx.quantize(_block(1.0, bad, 3.0), form)
        assert scales.tolist() == [255] and not codes.any()
        assert np.isnan(mx.dequantize(codes, scales, form)).all()


@pytest.mark.parametrize("form,half", [("mxfp4", 0.25), ("mxfp8", 2.0 ** -4)])
def test_error_of_a_rounding(form, half):
    """Within half a step of the element, or cut at the largest; quantizing the values again changes nothing."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 96)) * 2.0 ** rng.integers(-40, 40, (200, 1))
    codes, scales = mx.quantize(x, form)
    v = mx.dequantize(codes, scales, form)
    unit = np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)
    top = mx.MAGNITUDES[form][-1]
    inside = np.abs(x) <= top * unit
    low = mx.MAGNITUDES[form][1] * unit
    assert np.all(np.abs(v - x)[inside] <= np.maximum(half * np.abs(x), low / 2)[inside] * (1 + 1e-12))
    assert np.all(np.abs(v)[~inside] == (top * unit)[~inside])
    again = mx.quantize(v, form)
    assert np.array_equal(mx.dequantize(*again, form), v)


def test_planted_mistakes_are_seen():
    """Half-away rounding, the wrong order of two codes and a scale one too large each give other codes."""
    rng = np.random.default_rng(1)
    x = np.round(rng.standard_normal((4, 64)) * 4) / 8
    codes, scales = mx.quantize(x, "mxfp4")
    v = mx.dequantize(codes, scales, "mxfp4")
    assert not np.array_equal(mx.dequantize((codes >> 4) | (codes << 4), scales, "mxfp4"), v)
    assert not np.array_equal(mx.dequantize(codes, scales + 1, "mxfp4"), v)
    half = (mx.E2M1[1:] + mx.E2M1[:-1]) / 2
    a = np.abs(x.reshape(4, 2, 32)) / 2.0 ** (scales.astype(float)[..., None] - 127)
    away = np.searchsorted(half, a, side="right")
    assert np.any(away != mx.nearest(a, mx.E2M1))


def test_sums_beyond_the_bound_are_seen():
    """Sums rounded to binary16, or one element of a row off by a code, leave the bound that tests of the layer use."""
    rng = np.random.default_rng(2)
    x = mx.dequantize(*mx.quantize(rng.standard_normal((3, 256)), "mxfp8"), "mxfp8")
    W = mx.dequantize(*mx.quantize(rng.standard_normal((40, 256)), "mxfp4"), "mxfp4")
    y, tol = mx.mxfp4_linear(x, W, out_type="f32")
    assert np.any(np.abs(y.astype(np.float16) - y) > tol)
    W2 = W.copy()
    W2[:, 17] += 0.5 * np.abs(W).max() / 6
    assert np.any(np.abs(x @ W2.T - y) > tol)
    assert np.all(tol < 1e-2 * np.abs(x) @ np.abs(W).T)


def _sums_as_runs(parts, sizes, per):
    """How far sums may be off where neighbouring 128s of k, `per` of them, go to one sum each (132 roundings a 128)."""
    err, joined, joins = 0.0, 0.0, 0.0
    for first in range(0, len(parts), per):
        S = 0.0
        for part, size in zip(parts[first:first + per], sizes[first:first + per]):
            err += 132 * 2.0 ** -23 * (abs(S) + size)
            S += part
        joined += S
        joins += abs(joined)
    return err + (2.0 ** -24 * joins if per < len(parts) else 0.0)


@pytest.mark.parametrize("steps", [1, 3, 8, 9, 17, 28, 40])
def test_bound_of_sums_holds_for_runs_of_neighbours(steps):
    """A wave takes a run of neighbouring steps of k, an eighth or a fourth of them.  Where large parts of either sign lie at
    the two sides of a border between runs, the sums of the runs stay large while the running sum over all does not."""
    rng = np.random.default_rng(steps)
    x, W = np.zeros((6, 128 * steps)), np.zeros((1, 128 * steps))
    W[0, ::128] = 1.0
    for row in range(6):
        x[row, ::128] = rng.standard_normal(steps)
    for row, waves in enumerate((4, 8)):
        per = -(-steps // waves)
        x[row] = 0.0
        for border in range(per, steps, per):
            x[row, 128 * (border - 1)], x[row, 128 * border] = 1000.0, -1000.0
    bound = mx._sum_error(x, W)[1][:, 0]
    for row in range(6):
        parts = [float(x[row, 128 * k]) for k in range(steps)]
        for waves in (1, 4, 8):
            assert bound[row] >= _sums_as_runs(parts, [abs(p) for p in parts], -(-steps // waves)), (row, waves)
