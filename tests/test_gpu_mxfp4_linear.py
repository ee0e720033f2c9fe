"""GPU: the linear layer over MXFP4 weights (cq_mxfp4_linear) against its definition in 64 bits, within the bound that
oracle.microscaling.mxfp4_linear derives for each output."""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_amd as cq
from oracle import microscaling as mx
from parity import dev, say
from serving import TORCH, close, t16

pytestmark = pytest.mark.gpu


def _operands(rng, M, cols, inp, x="bf16", form="mxfp8", spread=2):
    """x's 16-bit values and the MXFP4 weights, with rows and blocks of different sizes."""
    xv = rng.standard_normal((M, inp)) * 2.0 ** rng.integers(-spread, spread + 1, (M, 1))
    xv[:, :: 37] *= 8
    xt, xn = t16(xv, x)
    wv = rng.standard_normal((cols, inp)) * 2.0 ** rng.integers(-spread, spread + 1, (cols, 1)) / np.sqrt(inp)
    codes, scales = mx.quantize(wv.astype(np.float32), "mxfp4")
    Q = mx.dequantize(*mx.quantize(xn, form), form)
    return xt, xn, Q, codes, scales, mx.dequantize(codes, scales, "mxfp4")


def _check(M, out, inp, x="bf16", form="mxfp8", y=None, act="none", gated=False, bias=False, res=False, ready=False,
           seed=0):
    say(f"mxfp4 linear: M={M} out={out} in={inp} {x} {form} ->{y or x} {act} gated={gated} bias={bias} res={res} ready={ready}")
    rng = np.random.default_rng(seed + M + out + inp)
    cols = 2 * out if gated else out
    xt, xn, Q, codes, scales, W = _operands(rng, M, cols, inp, x, form)
    bt, bn = t16(rng.standard_normal(cols), x) if bias else (None, None)
    rt, rn = t16(rng.standard_normal((M, out)), x) if res else (None, None)
    xs = None
    if ready:
        c, s = mx.quantize(xn, form)
        xt, xs = dev(c), dev(s)
    got = cq.mxfp4_linear(xt, dev(codes), dev(scales), x_scales=xs, x_format=form, bias=bt, residual=rt, activation=act,
                          gated=gated, out_dtype=TORCH[y or x])
    torch.cuda.synchronize()
    assert got.dtype == TORCH[y or x]
    want, tol = mx.mxfp4_linear(Q, W, bn, rn, act, gated, y or x)
    close(got, want, tol)


@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 33, 64, 65, 127, 130, 257, 520])
@pytest.mark.parametrize("out,inp", [(64, 128), (200, 384), (331, 1024)])
@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
def test_rows_and_shapes(M, out, inp, form):
    _check(M, out, inp, x="bf16" if M % 2 else "f16", form=form, y="f32", bias=True)


@pytest.mark.parametrize("out", [1, 2, 3, 7, 8, 15, 16, 17, 63, 65, 127, 129, 255, 256, 257])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_odd_widths(M, out):
    _check(M, out, 256, x="f16", form="mxfp4" if out % 2 else "mxfp8", res=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,x,y", [(1, "bf16", "bf16"), (5, "f16", "f32"), (96, "bf16", "f32"), (300, "f16", "f16")])
def test_epilogues(M, x, y, gated, act):
    _check(M, 136, 512, x, "mxfp8" if M % 2 else "mxfp4", y, act, gated, bias=True, res=True)


@pytest.mark.parametrize("ready", [False, True])
@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,out,inp", [(1, 1024, 3584), (4, 809, 4096), (203, 809, 4096), (200, 100, 4096),
                                       (1024, 1024, 1024), (700, 1030, 640)])
def test_larger(M, out, inp, form, ready):
    _check(M, out, inp, "bf16" if M % 2 else "f16", form, res=True, ready=ready)


@pytest.mark.parametrize("M,out,inp,kw", [
    (4100, 2060, 256, dict(bias=True, res=True)), (2049, 4095, 384, dict(y="f32", act="gelu")),
    (4097, 2046, 128, dict(x="f16", bias=True, act="silu", form="mxfp4")),
    (2050, 2200, 256, dict(gated=True, act="silu", bias=True, form="mxfp4")),
    (4200, 1037, 256, dict(x="f16", gated=True, act="gelu_tanh", res=True, y="f32")), (33000, 250, 128, dict(res=True)),
    (2048, 4096, 512, dict(x="f16", form="mxfp4")), (8200, 1025, 128, dict(act="relu", ready=True))])
def test_many_tiles(M, out, inp, kw):
    _check(M, out, inp, **kw)


@pytest.mark.parametrize("M,out,inp,kw", [
    (4100, 3100, 512, dict(form="mxfp4", bias=True, res=True)), (4100, 3104, 768, dict(form="mxfp4", y="f32")),
    (4097, 1553, 256, dict(form="mxfp4", gated=True, act="silu", bias=True, ready=True)),
    (4200, 3073, 1280, dict(x="f16", form="mxfp4", act="gelu", res=True)),
    (4100, 3104, 640, dict(form="mxfp4", bias=True)), (1100, 3100, 640, dict(form="mxfp8", res=True)),
    (1300, 2304, 1536, dict(form="mxfp8", bias=True, act="relu", ready=True)),
    (1025, 1160, 384, dict(x="f16", form="mxfp8", gated=True, act="gelu_tanh", res=True))])
def test_larger_tiles(M, out, inp, kw):
    """Tiles of 256 rows, rows of scales of whole and of odd lengths, steps of 256 and of 128, ends inside a tile."""
    _check(M, out, inp, **kw)


@pytest.mark.parametrize("M,out,inp", [(16, 4096, 256), (16, 4100, 256), (17, 4096, 256), (32, 8192, 128), (48, 5500, 128),
                                       (64, 4096, 128), (64, 4200, 128), (100, 4096, 128), (128, 8192, 128),
                                       (130, 8192, 128), (640, 4000, 128), (660, 4100, 128)])
@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
def test_either_side_of_the_borders_between_the_tiles(M, out, inp, form):
    _check(M, out, inp, x="f16" if M % 2 else "bf16", form=form, bias=True, y="f32")
    _check(M, out // 2, inp, form=form, gated=True, act="silu", ready=True)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("out,gated", [(14208, False), (7110, True), (24580, False), (12289, True)])
def test_few_rows_and_many_columns(M, out, gated):
    _check(M, out, 128, form="mxfp4" if M % 2 else "mxfp8", gated=gated, act="silu" if gated else "none", bias=True)


def test_zero_rows_or_columns():
    w, s = torch.zeros((0, 64), dtype=torch.uint8, device="cuda"), torch.zeros((0, 4), dtype=torch.uint8, device="cuda")
    x = torch.zeros((3, 128), dtype=torch.bfloat16, device="cuda")
    assert cq.mxfp4_linear(x, w, s).shape == (3, 0)
    w, s = torch.zeros((8, 64), dtype=torch.uint8, device="cuda"), torch.zeros((8, 4), dtype=torch.uint8, device="cuda")
    assert cq.mxfp4_linear(x[:0], w, s).shape == (0, 8)


@pytest.mark.parametrize("M", [1, 20, 300, 4200])
@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
def test_strided_and_in_place(M, form):
    """x, residual and y as strided rows; y over its residual."""
    rng = np.random.default_rng(M)
    out, inp = 260, 384
    xt, xn, Q, codes, scales, W = _operands(rng, M, out, inp, "bf16", form)
    wide = torch.full((M, inp + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + inp] = xt
    rt, rn = t16(rng.standard_normal((M, out)), "bf16")
    hold = torch.full((M, out + 7), 5.0, dtype=torch.bfloat16, device="cuda")
    hold[:, 3:3 + out] = rt
    y = hold[:, 3:3 + out]
    assert cq.mxfp4_linear(wide[:, 8:8 + inp], dev(codes), dev(scales), x_format=form, residual=y, out=y) is y
    torch.cuda.synchronize()
    want, tol = mx.mxfp4_linear(Q, W, None, rn)
    close(y, want, tol)
    assert (hold[:, :3] == 5).all() and (hold[:, 3 + out:] == 5).all()


@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M", [2, 40, 2100])
def test_same_result_from_values_and_from_codes(M, form):
    """The layer's own quantisation is mx_quantize's: both ways give the same bits."""
    x = torch.randn((M, 640), device="cuda").half()
    x[:, 5] *= 30
    w, s = cq.mx_quantize(torch.randn((1000, 640), device="cuda"), "mxfp4")
    codes, scales = cq.mx_quantize(x, form)
    a = cq.mxfp4_linear(x, w, s, x_format=form, out_dtype=torch.float32)
    b = cq.mxfp4_linear(codes, w, s, x_scales=scales, x_format=form, out_dtype=torch.float32)
    assert torch.equal(a, b)


@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M", [3, 600, 4100])
def test_infinities_nan_and_zeros(M, form):
    """A NaN or an infinity in x makes its row NaN, a NaN block of W its column; nothing else is touched."""
    x = torch.randn((M, 256), device="cuda").bfloat16()
    w, s = cq.mx_quantize(torch.randn((530, 256), device="cuda"), "mxfp4")
    clean = cq.mxfp4_linear(x, w, s, x_format=form, out_dtype=torch.float32)
    x[1, 77], x[2, 3] = float("nan"), -float("inf")
    s[7, 5] = 255
    y = cq.mxfp4_linear(x, w, s, x_format=form, out_dtype=torch.float32)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1:3], bad[:, 7] = True, True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])
    x.zero_()
    s[7, 5] = 127
    assert (cq.mxfp4_linear(x, w, s, x_format=form, out_dtype=torch.float32) == 0).all()


@pytest.mark.parametrize("M", [1, 300])
def test_scales_of_every_size(M):
    """Blocks of x from 2^-120 to 2^120 against blocks of W the other way round."""
    rng = np.random.default_rng(9)
    e = rng.integers(-120, 121, 8)
    xv = rng.standard_normal((M, 256)) * np.repeat(2.0 ** e, 32)
    wv = rng.standard_normal((70, 256)) * np.repeat(2.0 ** -e, 32)
    xt, xn = t16(xv, "bf16")
    codes, scales = mx.quantize(wv.astype(np.float32), "mxfp4")
    for form in ("mxfp4", "mxfp8"):
        got = cq.mxfp4_linear(xt, dev(codes), dev(scales), x_format=form, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want, tol = mx.mxfp4_linear(mx.dequantize(*mx.quantize(xn, form), form), mx.dequantize(codes, scales, "mxfp4"),
                                    out_type="f32")
        close(got, want, tol)


def test_streams_graph_and_workspace():
    """A captured call of many rows, replayed on new values, and one with a workspace of the caller's."""
    x = torch.randn((3000, 512), device="cuda").bfloat16()
    w, s = cq.mx_quantize(torch.randn((700, 512), device="cuda"), "mxfp4")
    need = cq.cq_mxfp4_linear_workspace_size(3000, 700, 512, 0, cq.MXFP8, 0)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = cq.mxfp4_linear(x, w, s, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(y, cq.mxfp4_linear(x, w, s))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = cq.mxfp4_linear(x, w, s)
        small = cq.mxfp4_linear(x[:3], w, s, x_format="mxfp4")
    for _ in range(4):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g, cq.mxfp4_linear(x, w, s))
        assert torch.equal(small, cq.mxfp4_linear(x[:3], w, s, x_format="mxfp4"))


def test_weights_past_32_bits():
    """Rows of W whose bytes lie beyond 2^32."""
    inp, cols = 1 << 17, (1 << 16) + 70
    w = torch.zeros((cols, inp // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((cols, inp // 32), 127, dtype=torch.uint8, device="cuda")
    w[-1, 5], w[3, 7] = 0x21, 0x07
    x = torch.randn((2, inp), device="cuda").bfloat16()
    y = cq.mxfp4_linear(x, w, s, x_format="mxfp8", out_dtype=torch.float32)
    q = cq.mx_dequantize(*cq.mx_quantize(x, "mxfp8"), "mxfp8", torch.float32)
    assert torch.equal(y[:, -1], 0.5 * q[:, 10] + q[:, 11]) and torch.equal(y[:, 3], 6 * q[:, 14])
    assert not y[:, 4:-1].any()


@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,out,gated", [(3, 40, False), (70, 520, True), (300, 8320, False)])
def test_rows_far_apart(M, out, gated, form):
    """Codes, their scales, residual and result with rows 2^23 bytes or elements apart: as with rows one behind the other."""
    g = torch.Generator(device="cuda").manual_seed(2)
    apart, inp = 1 << 23, 512
    w, s = cq.mx_quantize(torch.randn((out * (2 if gated else 1), inp), generator=g, device="cuda"), "mxfp4")
    x, e = cq.mx_quantize(torch.randn((M, inp), generator=g, device="cuda"), form)
    r = torch.randn((M, out), generator=g, device="cuda").bfloat16()

    def far(t):
        v = torch.empty((M, apart), dtype=t.dtype, device="cuda")[:, : t.shape[1]]
        return v.copy_(t)

    kw = dict(x_format=form, gated=gated, activation="silu" if gated else "none")
    want = cq.mxfp4_linear(x, w, s, x_scales=e, residual=r, **kw)
    y = far(torch.full_like(r, 9.0))
    cq.mxfp4_linear(far(x), w, s, x_scales=far(e), residual=far(r), out=y, **kw)
    assert torch.equal(y, want)
    assert torch.equal(cq.mxfp4_linear(far(x), w, s, x_scales=e, out=far(r), residual=r, **kw), want)


@pytest.mark.parametrize("M,out", [(5, 70), (130, 700), (300, 8320)])
def test_nan_codes(M, out):
    """An element of x that is NaN makes its row NaN, and no other."""
    g = torch.Generator(device="cuda").manual_seed(4)
    w, s = cq.mx_quantize(torch.randn((out, 256), generator=g, device="cuda"), "mxfp4")
    x, e = cq.mx_quantize(torch.randn((M, 256), generator=g, device="cuda"), "mxfp8")
    clean = cq.mxfp4_linear(x, w, s, x_scales=e, out_dtype=torch.float32)
    for row, k, code in ((0, 255, 0x7F), (M - 1, 3, 0xFF), (M // 2, 130, 0x7F)):
        bad = x.clone()
        bad[row, k] = code
        y = cq.mxfp4_linear(bad, w, s, x_scales=e, out_dtype=torch.float32)
        assert torch.isnan(y[row]).all()
        others = torch.arange(M, device="cuda") != row
        assert torch.equal(y[others], clean[others])


@pytest.mark.parametrize("M,out,gated", [(1, 16448, False), (8, 24600, False), (9, 16448, False), (1, 41024, False),
                                         (8, 20520, True), (16, 41027, False), (16, 20513, True), (17, 41024, False)])
@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
def test_codes_of_few_rows_and_many_columns(M, out, gated, form):
    _check(M, out, 128, form=form, gated=gated, act="silu" if gated else "none", bias=True, ready=True)


@pytest.mark.parametrize("M,form", [(1, "mxfp4"), (8, "mxfp4"), (1, "mxfp8"), (5, "mxfp8"), (8, "mxfp8"), (16, "mxfp8")])
def test_few_rows_have_the_same_sums_from_values_and_from_codes(M, form):
    """Through many columns as well: up to 8 rows (MXFP8: 16) are multiplied alike, in the same order."""
    g = torch.Generator(device="cuda").manual_seed(M)
    xt = torch.randn((M, 2048), generator=g, device="cuda").bfloat16()
    w, s = cq.mx_quantize(torch.randn((41024, 2048), generator=g, device="cuda"), "mxfp4")
    c, e = cq.mx_quantize(xt, form)
    a = cq.mxfp4_linear(xt, w, s, x_format=form, out_dtype=torch.float32)
    b = cq.mxfp4_linear(c, w, s, x_scales=e, x_format=form, out_dtype=torch.float32)
    assert torch.equal(a, b)
