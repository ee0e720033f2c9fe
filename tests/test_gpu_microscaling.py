"""GPU: microscaled blocks of rows and of a paged cache (cq_mx_quantize, cq_mx_dequantize, cq_kv_cache_write_mx), bit by
bit against their definition."""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_amd as cq
from oracle import microscaling as mx
from parity import dev, say
from serving import TORCH, i32, t16

pytestmark = pytest.mark.gpu

FORMS = ["mxfp4", "mxfp8"]


def _same(got, want, label=""):
    got = got.cpu().numpy()
    assert got.shape == want.shape and got.dtype == want.dtype, label
    assert np.array_equal(got, want), f"{label}: {np.sum(got != want)} of {want.size} differ, first at {np.argwhere(got != want)[:3]}"


def _check(x, form, label=""):
    """x a device tensor: its codes and scales, and the values read back in every type."""
    codes, scales = cq.mx_quantize(x, form)
    torch.cuda.synchronize()
    wc, ws = mx.quantize(x.double().cpu().numpy(), form)
    _same(scales, ws, label + " scales")
    _same(codes, wc, label + " codes")
    want = mx.dequantize(wc, ws, form)
    for dt in TORCH.values():
        y = cq.mx_dequantize(codes, scales, form, out_dtype=dt)
        torch.cuda.synchronize()
        w, y = torch.from_numpy(want).to(dt), y.cpu()
        assert y.dtype == dt and torch.equal(torch.isnan(y), torch.isnan(w))
        assert torch.equal(y.masked_fill(torch.isnan(y), 0), w.masked_fill(torch.isnan(w), 0)), f"{label} {dt}"


def _patterns(kind):
    """Every value of a 16-bit type, an infinity or a NaN only in blocks of their own, at their own neighbours' scale and
    beside a large and a small one."""
    bits = np.arange(65536, dtype=np.uint16)
    v = torch.from_numpy(bits.view(np.int16)).view(TORCH[kind])
    near = v.view(-1, 32)
    rng = np.random.default_rng(3)
    mixed = v[torch.from_numpy(rng.permutation(65536))].view(-1, 32)
    finite = torch.where(torch.isfinite(mixed), mixed, torch.zeros_like(mixed))
    stair = v.view(256, 256).t().contiguous().view(-1, 32)  # neighbours 256 patterns apart
    return torch.cat([near, finite, stair, mixed])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_every_16_bit_value(form, kind):
    say(f"mx patterns {form} {kind}")
    _check(_patterns(kind).cuda(), form, kind)


@pytest.mark.parametrize("form", FORMS)
def test_fp32_values_of_every_size(form):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((400, 320)) * 2.0 ** rng.integers(-60, 60, (400, 320))
    y = rng.standard_normal((400, 320)) * 2.0 ** rng.integers(-150, 127, (400, 1))
    y[3, 40] = np.nan
    y[5, 64] = -np.inf
    y[7] = 0
    ties = rng.integers(-4096, 4097, (400, 320)) / 128.0  # ties between elements at many scales
    with np.errstate(over="ignore"):
        a = np.concatenate([x, y, ties]).astype(np.float32)
    _check(dev(a), form, "fp32")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (7, 96), (1, 2080), (129, 160), (2, 3, 5, 224), (1000, 32), (0, 64)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_shapes(form, shape, kind):
    x = torch.randn(shape, device="cuda").to(TORCH[kind])
    _check(x, form, str(shape))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strided_rows(form, kind):
    x = torch.randn((37, 400), device="cuda").to(TORCH[kind])[:, 16:208]
    assert not x.is_contiguous()
    _check(x, form, "strided")
    codes, scales = cq.mx_quantize(x.contiguous(), form)
    wide = torch.full((37, codes.shape[1] + 32), 0xEE, dtype=torch.uint8, device="cuda")
    wides = torch.full((37, scales.shape[1] + 3), 0xEE, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + codes.shape[1]] = codes
    wides[:, 1:1 + scales.shape[1]] = scales
    a = cq.mx_dequantize(wide[:, 16:16 + codes.shape[1]], wides[:, 1:1 + scales.shape[1]], form, torch.float32)
    assert torch.equal(a, cq.mx_dequantize(codes, scales, form, torch.float32))


@pytest.mark.parametrize("form", FORMS)
def test_every_code_at_every_scale(form):
    """All 256 bytes at all 256 scales, read back in every type: rounded once, NaN for 255 and e4m3's NaN codes."""
    bytes_ = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    blocks = 256 * (2 if form == "mxfp4" else 1) // 32
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], blocks, 1)
    want = mx.dequantize(bytes_, scales, form)
    for dt in TORCH.values():
        y = cq.mx_dequantize(dev(bytes_), dev(scales), form, out_dtype=dt).cpu()
        with np.errstate(over="ignore"):
            w = torch.from_numpy(want).to(dt)
        assert torch.equal(torch.isnan(y), torch.isnan(w))
        assert torch.equal(y.masked_fill(torch.isnan(y), 0), w.masked_fill(torch.isnan(w), 0)), dt


def test_larger_than_32_bits_of_bytes():
    """More than 2^32 bytes of values: offsets past 32 bits; the last rows are those of a call of their own."""
    x = torch.randn((1 << 20, 32), device="cuda").bfloat16().repeat(66, 1)  # 2.2e9 values, 4.4 GB
    x[-5:] *= 3
    codes, scales = cq.mx_quantize(x, "mxfp8")
    y = cq.mx_dequantize(codes, scales, "mxfp8")
    c, e = cq.mx_quantize(x[-4096:], "mxfp8")
    assert torch.equal(codes[-4096:], c) and torch.equal(scales[-4096:], e)
    assert torch.equal(y[-4096:], cq.mx_dequantize(c, e, "mxfp8")) and torch.equal(y[1 << 26 : (1 << 26) + 99], y[:99])


# ---------------------------------------------------------------- the cache
def _write(T, Hkv, D, page, form, kind, seed=0, order="hnd", packed=True, slots=None, n_pages=None):
    say(f"cache write mx T={T} Hkv={Hkv} D={D} page={page} {form} {kind} {order}")
    rng = np.random.default_rng(seed)
    n_pages = -(-T // page) + 2 if n_pages is None else n_pages
    if packed:
        rows, values = t16(rng.standard_normal((T, 3 * Hkv, D)) * 2.0 ** rng.integers(-6, 6, (T, 3 * Hkv, 1)), kind)
        k, v, kn, vn = rows[:, Hkv:2 * Hkv], rows[:, 2 * Hkv:], values[:, Hkv:2 * Hkv], values[:, 2 * Hkv:]
    else:  # nothing aligned: an odd offset and odd strides
        flat, values = t16(rng.standard_normal(2 * T * Hkv * (D + 1) + 1), kind)
        k, v = flat[1:].view(2, T, Hkv, D + 1)[:, :, :, :D].unbind(0)
        kn, vn = values[1:].reshape(2, T, Hkv, D + 1)[:, :, :, :D]
    if slots is None:
        slots = rng.permutation(n_pages * page)[:T]
    width = D // 2 if form == "mxfp4" else D
    shape = (n_pages, Hkv, page) if order == "hnd" else (n_pages, page, Hkv)
    caches = [torch.full(shape + (w,), 0xA5, dtype=torch.uint8, device="cuda") for w in (width, D // 32, width, D // 32)]
    seen = caches if order == "hnd" else [c.transpose(1, 2) for c in caches]
    cq.kv_cache_write_mx(k, v, *seen, i32(slots))
    torch.cuda.synchronize()
    for at, (values, name) in enumerate(((kn, "k"), (vn, "v"))):
        codes, scales = mx.quantize(values, form)
        for got, rows, what in ((seen[2 * at], codes, "codes"), (seen[2 * at + 1], scales, "scales")):
            want = np.full(tuple(got.shape), 0xA5, np.uint8)
            for t, s in enumerate(np.asarray(slots)):
                if 0 <= s < n_pages * page:
                    want[s // page, :, s % page] = rows[t]
            _same(got.contiguous(), want, f"{name} {what}")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 32, 1), (1, 2, 128, 16), (33, 4, 64, 8), (50, 3, 96, 24), (17, 1, 256, 7),
                                          (300, 8, 128, 16), (9, 5, 160, 3), (12, 2, 224, 64), (70, 2, 192, 32)])
def test_cache_write(form, kind, T, Hkv, D, page):
    _write(T, Hkv, D, page, form, kind)


@pytest.mark.parametrize("form", FORMS)
def test_cache_write_orders_and_alignment(form):
    _write(40, 3, 64, 16, form, "bf16", order="nhd")
    _write(40, 3, 96, 5, form, "f16", order="nhd", packed=False)
    _write(40, 2, 128, 16, form, "bf16", packed=False)


@pytest.mark.parametrize("form", FORMS)
def test_cache_write_skips_what_has_no_slot(form):
    _write(6, 2, 64, 4, form, "bf16", slots=[5, -1, 12, 1 << 30, 0, -(1 << 31)], n_pages=3)
    _write(3, 1, 32, 4, form, "f16", slots=[-1, -1, -1], n_pages=1)


@pytest.mark.parametrize("form", FORMS)
def test_cache_write_of_infinities_and_nan(form):
    k = torch.randn((4, 2, 64), device="cuda").bfloat16()
    k[1, 0, 5], k[2, 1, 40], k[3, 0, 33] = float("nan"), float("inf"), -float("inf")
    caches = [torch.zeros((1, 2, 4, w), dtype=torch.uint8, device="cuda") for w in (64 if form == "mxfp8" else 32, 2) * 2]
    cq.kv_cache_write_mx(k, -k, *caches, i32(np.arange(4)))
    for at, values in ((0, k), (2, -k)):
        codes, scales = mx.quantize(values.double().cpu().numpy(), form)
        _same(caches[at][0].transpose(0, 1).contiguous(), codes)
        _same(caches[at + 1][0].transpose(0, 1).contiguous(), scales)
    assert (caches[1] == 255).sum() == 3


@pytest.mark.parametrize("form", FORMS)
def test_cache_past_32_bits(form):
    """A page whose bytes lie beyond 2^32."""
    D, page = 256, 64
    n_pages = (1 << 32) // (page * D // (2 if form == "mxfp4" else 1)) + 40
    caches = [torch.zeros((n_pages, 1, page, w), dtype=torch.uint8, device="cuda")
              for w in (D // (2 if form == "mxfp4" else 1), D // 32) * 2]
    k = torch.randn((2, 1, D), device="cuda").half()
    last = n_pages * page - 1
    cq.kv_cache_write_mx(k, k, *caches, i32([last, 3]))
    codes, scales = cq.mx_quantize(k, form)
    for c, want in zip(caches, (codes, scales, codes, scales)):
        assert torch.equal(c[-1, :, -1], want[0]) and torch.equal(c[0, :, 3], want[1])
        assert int(c.count_nonzero()) == int(want.count_nonzero())


def test_streams_and_graphs():
    """On a side stream, and replayed from a graph with other inputs in between."""
    x = torch.randn((64, 256), device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    codes, scales = cq.mx_quantize(x, "mxfp4", stream=side)
    y = cq.mx_dequantize(codes, scales, "mxfp4", stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, cq.mx_dequantize(*cq.mx_quantize(x, "mxfp4"), "mxfp4"))
    k = torch.randn((8, 2, 64), device="cuda").bfloat16()
    caches = [torch.zeros((2, 2, 8, w), dtype=torch.uint8, device="cuda") for w in (64, 2, 64, 2)]
    slots = i32(np.arange(8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        cq.mx_quantize(x, "mxfp8")
        cq.kv_cache_write_mx(k, k, *caches, slots)
    side.synchronize()
    with torch.cuda.graph(graph):
        gc, gs = cq.mx_quantize(x, "mxfp8")
        gy = cq.mx_dequantize(gc, gs, "mxfp8")
        cq.kv_cache_write_mx(k, k, *caches, slots)
    for i in range(4):
        x.normal_()
        k.normal_(std=2.0 ** i)
        slots.copy_(i32(np.random.default_rng(i).permutation(16)[:8]))
        for c in caches:
            c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, cq.mx_dequantize(*cq.mx_quantize(x, "mxfp8"), "mxfp8"))
        fresh = [torch.zeros_like(c) for c in caches]
        cq.kv_cache_write_mx(k, k, *fresh, slots)
        assert all(torch.equal(a, b) for a, b in zip(caches, fresh))
