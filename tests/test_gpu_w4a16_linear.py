"""GPU: the linear layer over GPTQ-v1 tensors (cq_w4a16_linear) against its definition in 64 bits, within the
bound that oracle.serving.w4a16_linear derives for each output."""
import numpy as np
import pytest
import torch

import oracle
import post_weight_quantization_group_amd as cq
from oracle import serving as ref
from parity import dev, say
from serving import TORCH, close, t16

pytestmark = pytest.mark.gpu


def _weights(rng, cols, inp):
    codes = rng.integers(-8, 8, (cols, inp)).astype(np.int8)
    sv = rng.uniform(1e-3, 2e-2, (cols, inp // 128)).astype(np.float16)
    return oracle.pack_gptq_v1(codes, sv.view(np.uint16), cols, inp)


def _check(M, out, inp, x="bf16", y=None, act="none", gated=False, bias=False, res=False, seed=0, offset=0.0):
    say(f"linear: M={M} out={out} in={inp} {x}->{y or x} {act} gated={gated} bias={bias} res={res}")
    rng = np.random.default_rng(seed + M + out + inp)
    cols = 2 * out if gated else out
    qw, sc = _weights(rng, cols, inp)
    xt, xn = t16(rng.standard_normal((M, inp)) + offset, x)
    bt, bn = t16(rng.standard_normal(cols), x) if bias else (None, None)
    rt, rn = t16(rng.standard_normal((M, out)), x) if res else (None, None)
    got = cq.w4a16_linear(xt, dev(qw), dev(sc.view(np.int16)), bias=bt, residual=rt, activation=act, gated=gated,
                          out_dtype=TORCH[y or x])
    torch.cuda.synchronize()
    assert got.dtype == TORCH[y or x]
    want, tol = ref.w4a16_linear(xn, qw, sc, bn, rn, act, gated, y or x)
    close(got, want, tol)


@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 33, 64, 65, 127, 130, 257, 520])
@pytest.mark.parametrize("out,inp", [(64, 128), (200, 384), (331, 1024)])
def test_rows_and_shapes(M, out, inp):
    _check(M, out, inp, x="bf16" if M % 2 else "f16", y="f32", bias=True)


@pytest.mark.parametrize("out", [1, 2, 3, 7, 8, 15, 16, 17, 63, 65, 127, 129, 255, 256, 257])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_odd_widths(M, out):
    _check(M, out, 256, x="f16", res=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,x,y", [(1, "bf16", "bf16"), (5, "f16", "f32"), (96, "bf16", "f32"), (300, "f16", "f16")])
def test_epilogues(M, x, y, gated, act):
    _check(M, 136, 512, x, y, act, gated, bias=True, res=True)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,out", [(1, 500), (40, 500), (16500, 120)])
def test_tails_of_the_activations(M, out, gated, act):
    """x = 0, so the bias alone: arguments down to where an fp32 value of the activation is no longer a normal number
    keep their relative accuracy."""
    rng = np.random.default_rng(out)
    cols = 2 * out if gated else out
    qw, sc = _weights(rng, cols, 128)
    z = np.linspace(-11.5 if act == "gelu" else -9.0 if act == "gelu_tanh" else -80.0, 6.0, out)
    bt, bn = t16(np.concatenate([z, np.full(out, 3.0)]) if gated else z, "bf16")
    got = cq.w4a16_linear(torch.zeros((M, 128), dtype=torch.bfloat16, device="cuda"), dev(qw), dev(sc.view(np.int16)),
                          bias=bt, activation=act, gated=gated, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, tol = ref.w4a16_linear(np.zeros((M, 128)), qw, sc, bn, None, act, gated, "f32")
    assert np.all(tol[want != 0] <= 2.0 ** -10 * np.abs(want[want != 0]))
    close(got, want, tol)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 16500])
def test_activations_of_infinity_and_nan(M, act):
    qw, sc = _weights(np.random.default_rng(1), 4 * 32, 128)
    bias = torch.tensor([np.inf, np.nan, 60000.0, 3e38] * 32, device="cuda").bfloat16()
    y = cq.w4a16_linear(torch.zeros((M, 128), dtype=torch.bfloat16, device="cuda"), dev(qw), dev(sc.view(np.int16)),
                        bias=bias, activation=act, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert (y[:, 0::4] == np.inf).all() and torch.isnan(y[:, 1::4]).all()
    assert torch.equal(y[:, 2::4], bias[2::4].float().expand(M, -1)) and (y[:, 3::4] > 2.9e38).all()


@pytest.mark.parametrize("M,out,inp", [(1, 1024, 3584), (4, 809, 4096), (200, 100, 4096), (1024, 1024, 1024),
                                       (700, 1030, 640)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_larger(M, out, inp, x):
    _check(M, out, inp, x, res=True)


@pytest.mark.parametrize("M,out,inp,kw", [
    (4100, 2060, 256, dict(bias=True, res=True)), (2049, 4095, 384, dict(y="f32", act="gelu")),
    (4097, 2046, 128, dict(x="f16", bias=True, act="silu")), (2050, 2200, 256, dict(gated=True, act="silu", bias=True)),
    (4200, 1037, 256, dict(x="f16", gated=True, act="gelu_tanh", res=True, y="f32")), (33000, 250, 128, dict(res=True)),
    (2048, 4096, 512, dict(x="f16")), (8200, 1025, 128, dict(act="relu"))])
def test_many_tiles(M, out, inp, kw):
    _check(M, out, inp, **kw)


@pytest.mark.parametrize("M", [1280, 1281, 1408, 1409])
@pytest.mark.parametrize("out,gated", [(2048, False), (1001, True), (1030, True), (2047, False)])
def test_either_side_of_the_border_between_the_kernels(M, out, gated):
    _check(M, out, 128, x="f16" if M % 2 else "bf16", gated=gated, act="silu", bias=True, res=True)


@pytest.mark.parametrize("M,out", [(1920, 896), (1921, 896), (2048, 889), (2304, 3456), (2305, 3456), (2433, 3449)])
@pytest.mark.parametrize("gated", [False, True])
def test_tiles_of_either_width(M, out, gated):
    out = out // 2 if gated else out
    _check(M, out, 384, x="bf16" if M % 2 else "f16", gated=gated, act="gelu", bias=True, y="f32" if gated else None)


@pytest.mark.parametrize("M", [1, 32, 33, 64, 65])
@pytest.mark.parametrize("out,gated", [(14208, False), (14209, False), (14212, False), (7110, True), (24576, False),
                                       (24580, False), (12289, True), (12290, True)])
def test_few_rows_and_many_columns(M, out, gated):
    """Either side of the borders between the kernels at few rows: 111 and 112 tiles, 192 and 193."""
    _check(M, out, 128, x="f16" if M % 2 else "bf16", gated=gated, act="silu", res=True)


@pytest.mark.parametrize("M", [1, 16])
def test_few_rows_do_not_pay_for_128(M):
    """Few rows through a wide layer take the kernel that reads its words and little else."""
    qw = torch.randint(-2 ** 31, 2 ** 31 - 1, (512, 16384), device="cuda").int()
    sc = torch.rand((32, 16384), device="cuda").half()
    x = torch.randn((128, 4096), device="cuda").bfloat16()
    y = torch.empty((128, 16384), device="cuda").bfloat16()

    def least(m):
        times = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(20):
                cq.w4a16_linear(x[:m], qw, sc, out=y[:m])
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    few, many = least(M), least(128)
    say(f"linear: {M} rows {50 * few:.1f} us, 128 rows {50 * many:.1f}")
    assert few < 0.5 * many


@pytest.mark.parametrize("M,out", [(1, 64), (30, 33), (300, 65), (4100, 2060), (2049, 4097)])
@pytest.mark.parametrize("gated", [False, True])
def test_scales_of_zero_and_of_every_size(M, out, gated):
    """Groups whose scale is 0 (with any codes) among scales from the smallest binary16 value to large ones,
    of either sign."""
    rng = np.random.default_rng(M + out)
    cols, inp = 2 * out if gated else out, 1024
    codes = rng.integers(-8, 8, (cols, inp)).astype(np.int8)
    sv = (2.0 ** rng.uniform(-24, 4, (cols, 8)) * rng.choice([-1, 1], (cols, 8))).astype(np.float16)
    sv[rng.random((cols, 8)) < 0.3] = 0
    sv[::7, 0], sv[::5, 7], sv[::11], sv[1::11] = 0, 0, 0, np.float16(2.0 ** -24)
    qw, sc = oracle.pack_gptq_v1(codes, sv.view(np.uint16), cols, inp)
    xt, xn = t16(rng.standard_normal((M, inp)), "bf16")
    got = cq.w4a16_linear(xt, dev(qw), dev(sc.view(np.int16)), gated=gated, out_dtype=torch.float32)
    torch.cuda.synchronize()
    close(got, *ref.w4a16_linear(xn, qw, sc, gated=gated, out_type="f32"))


@pytest.mark.parametrize("M,out,gated", [(2048, 1030, False), (2048, 1024, False), (2100, 515, True), (2048, 512, True),
                                         (16, 14400, False), (3, 9000, True)])
def test_such_scales_at_other_tiles(M, out, gated):
    """128 columns a workgroup, and few rows of many columns."""
    test_scales_of_zero_and_of_every_size(M, out, gated)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_rows_with_a_common_offset(M):
    """All activations near 3: the row's sum is 100 times its entries' spread."""
    _check(M, 72, 512, y="f32", offset=3.0)


@pytest.mark.parametrize("M", [1, 24, 200, 33000])
def test_strided_rows_and_residual_in_place(M):
    rng = np.random.default_rng(M)
    out, inp = 72, 256
    qw, sc = _weights(rng, out, inp)
    xt, xn = t16(rng.standard_normal((M, inp + 64)), "bf16")
    rt, rn = t16(rng.standard_normal((M, out + 9)), "bf16")
    view, rest = rt[:, 5:5 + out], rt.clone()
    cq.w4a16_linear(xt[:, 16:16 + inp], dev(qw), dev(sc.view(np.int16)), residual=view, out=view)
    torch.cuda.synchronize()
    want, tol = ref.w4a16_linear(xn[:, 16:16 + inp], qw, sc, None, rn[:, 5:5 + out])
    close(view, want, tol)
    assert torch.equal(rt[:, :5], rest[:, :5]) and torch.equal(rt[:, 5 + out:], rest[:, 5 + out:])


@pytest.mark.parametrize("M", [3, 40, 300, 33000])
def test_a_row_of_nan_or_infinity_stays_in_its_row(M):
    rng = np.random.default_rng(M)
    qw, sc = _weights(rng, 80, 256)
    x = rng.standard_normal((M, 256))
    x[1, 7], x[M - 1, 200] = np.nan, np.inf
    xt, xn = t16(x, "bf16")
    got = cq.w4a16_linear(xt, dev(qw), dev(sc.view(np.int16)))
    torch.cuda.synchronize()
    clean = [m for m in range(M) if m not in (1, M - 1)]
    want, tol = ref.w4a16_linear(xn[clean], qw, sc)
    close(got[clean], want, tol)
    assert torch.isnan(got[1]).all()
    codes = oracle.unpack_gptq_v1(qw, sc)[0][:, 200]
    last = got[M - 1].float().cpu().numpy()
    assert np.all(np.isnan(last[codes == 0])) and np.all(~np.isfinite(last))


def test_memory_behind_the_last_row_and_column_is_left_alone():
    rng = np.random.default_rng(9)
    for M, out in ((1, 33), (17, 65), (130, 129), (300, 200), (2100, 4001)):
        qw, sc = _weights(rng, out, 128)
        xt, xn = t16(rng.standard_normal((M, 128)), "f16")
        buf = torch.full((M + 140, out + 140), 5.0, dtype=torch.float32, device="cuda")
        cq.w4a16_linear(xt, dev(qw), dev(sc.view(np.int16)), out=buf[:M, :out])
        torch.cuda.synchronize()
        close(buf[:M, :out], *ref.w4a16_linear(xn, qw, sc, out_type="f32"))
        assert (buf[M:] == 5).all() and (buf[:M, out:] == 5).all()


def test_repeated_calls_and_another_stream_give_the_same_bits():
    rng = np.random.default_rng(4)
    for M in (1, 100, 600, 33000):
        qw, sc = (dev(a) for a in _weights(rng, 200, 1024))
        xt, _ = t16(rng.standard_normal((M, 1024)), "bf16")
        a = cq.w4a16_linear(xt, qw, sc.view(torch.int16), activation="gelu")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        b = cq.w4a16_linear(xt, qw, sc.view(torch.int16), activation="gelu", stream=s)
        s.synchronize()
        assert torch.equal(a, b)


def test_matches_the_consumer_check():
    """cq_w4a16_matmul of the same tensors: both within their bounds of the definition, so within their sum."""
    rng = np.random.default_rng(6)
    qw, sc = _weights(rng, 96, 512)
    xt, xn = t16(rng.standard_normal((50, 512)), "bf16")
    a = cq.w4a16_matmul(xt, dev(qw), dev(sc.view(np.int16)))
    b = cq.w4a16_linear(xt, dev(qw), dev(sc.view(np.int16)), out_dtype=torch.float32)
    torch.cuda.synchronize()
    tol = ref.w4a16_linear(xn, qw, sc, out_type="f32")[1]
    close(b, a.double().cpu().numpy(), 2 * tol)


def test_replayed_graph():
    rng = np.random.default_rng(8)
    qw, sc = (dev(a) for a in _weights(rng, 256, 512))
    sc = sc.view(torch.int16)
    for M in (1, 300, 33000):
        xt, _ = t16(rng.standard_normal((M, 512)), "f16")
        out = torch.empty((M, 256), dtype=torch.float16, device="cuda")
        cq.w4a16_linear(xt, qw, sc, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cq.w4a16_linear(xt, qw, sc, out=out)
        for k in range(4):
            xt.copy_(t16(rng.standard_normal((M, 512)), "f16")[0])
            eager = cq.w4a16_linear(xt, qw, sc)
            out.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager), (M, k)


def test_refusals():
    qw = torch.zeros((16, 8), dtype=torch.int32, device="cuda")
    sc = torch.zeros((1, 8), dtype=torch.int16, device="cuda")
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(x=x.float()), dict(x=x[:, :64]), dict(qweight=qw[:8]), dict(scales=sc[:, :4]),
               dict(bias=torch.zeros(7, dtype=x.dtype, device="cuda")), dict(bias=torch.zeros(8, device="cuda")),
               dict(residual=torch.zeros((2, 8), dtype=torch.float16, device="cuda")), dict(activation="tanh"),
               dict(out_dtype=torch.float16), dict(out=torch.zeros((2, 7), device="cuda")), dict(x=x.cpu()),
               dict(x=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            cq.w4a16_linear(**dict(dict(x=x, qweight=qw, scales=sc), **kw))
    wide = torch.zeros((2, 140), dtype=torch.bfloat16, device="cuda")
    for bad in (wide[:, 4:132], torch.zeros((2, 129), dtype=torch.bfloat16, device="cuda")[:, :128]):
        with pytest.raises(cq.CQError):                       # rows not 16-byte aligned
            cq.w4a16_linear(bad, qw, sc)
    assert cq.w4a16_linear(x[:0], qw, sc).shape == (0, 8)
