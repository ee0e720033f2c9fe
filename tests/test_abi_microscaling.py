"""The microscaled formats' C entry points and helpers without a GPU: bad arguments are refused before anything reaches
HIP."""
import pytest
import torch

import post_weight_quantization_group_amd as cq

FAKE = 1 << 20  # a 16-byte-aligned address that is never dereferenced: every call below fails its checks


def _rows(entry, **kw):
    a = dict(x=FAKE, ldx=128, xt=cq.BF16, rows=4, len=128, form=cq.MXFP4, codes=FAKE, ldc=64, scales=FAKE, lds=4)
    a.update(kw)
    lib = cq.load()
    if entry == "quantize":
        return lib.cq_mx_quantize(a["x"], a["ldx"], a["xt"], a["rows"], a["len"], a["form"], a["codes"], a["ldc"],
                                  a["scales"], a["lds"], None)
    return lib.cq_mx_dequantize(a["codes"], a["ldc"], a["scales"], a["lds"], a["form"], a["rows"], a["len"], a["x"],
                                a["ldx"], a["xt"], None)


@pytest.mark.parametrize("entry", ["quantize", "dequantize"])
@pytest.mark.parametrize("kw", [
    dict(xt=3), dict(xt=-1), dict(form=2), dict(form=5), dict(rows=-1), dict(len=0), dict(len=-32), dict(len=48),
    dict(len=1 << 34, ldx=1 << 34, ldc=1 << 33, lds=1 << 29), dict(rows=1 << 27), dict(rows=1 << 62), dict(x=None),
    dict(codes=None), dict(scales=None), dict(x=FAKE + 8), dict(codes=FAKE + 8), dict(ldx=120), dict(ldx=132),
    dict(ldc=48), dict(ldc=72), dict(lds=3), dict(form=cq.MXFP8),
])
def test_rows_reject_before_launch(entry, kw):
    assert _rows(entry, **kw) == -1


@pytest.mark.parametrize("entry", ["quantize", "dequantize"])
def test_no_rows_are_a_no_op(entry):
    assert _rows(entry, rows=0, x=None, codes=None, scales=None) == 0


def _cache(**kw):
    a = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, page_stride=2048, head_stride=1024, row_stride=64,
             scale_page_stride=64, scale_head_stride=32, scale_row_stride=2, format=cq.MXFP8, n_pages=9, page_size=16,
             kv_heads=2, head_dim=64)
    a.update({k: v for k, v in kw.items() if k in a})
    return cq.MxCache(**a)


def _write(**kw):
    a = dict(k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, type=cq.BF16, slots=FAKE, T=3)
    a.update({k: v for k, v in kw.items() if k in a})
    return cq.load().cq_kv_cache_write_mx(a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["type"],
                                          None if kw.get("cache", 1) is None else _cache(**kw), a["slots"], a["T"], None)


BAD_CACHES = [dict(format=0), dict(format=5), dict(n_pages=-1), dict(page_size=0), dict(kv_heads=0), dict(head_dim=0),
              dict(head_dim=80), dict(head_dim=288), dict(page_stride=-16), dict(head_stride=1000), dict(row_stride=8),
              dict(scale_row_stride=-1), dict(scale_page_stride=-1), dict(k_codes=FAKE + 8), dict(v_codes=FAKE + 4)]


@pytest.mark.parametrize("kw", BAD_CACHES + [
    dict(cache=None), dict(type=cq.F32), dict(T=-1), dict(kt=-1), dict(vh=-2), dict(k=None), dict(v=None),
    dict(k_codes=None), dict(v_codes=None), dict(k_scales=None), dict(v_scales=None), dict(slots=None), dict(k=FAKE + 1),
    dict(v=FAKE + 1), dict(slots=FAKE + 2), dict(T=1 << 27), dict(T=(1 << 31) - 1, kv_heads=1 << 20),
])
def test_cache_write_rejects_before_launch(kw):
    assert _write(**kw) == -1


def test_cache_write_of_nothing_is_a_no_op():
    assert _write(T=0, k=None) == 0 and _write(n_pages=0, k_codes=None, k_scales=None) == 0


def _refused(match, call, *args, **kw):
    with pytest.raises(ValueError, match=match):
        call(*args, **kw)


def test_helpers_refuse():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    _refused("format", cq.mx_quantize, x, "mxfp6")
    _refused("multiple of 32", cq.mx_quantize, x[:, :48], "mxfp4")
    _refused("multiple of 32", cq.mx_quantize, x[:, :0], "mxfp4")
    _refused("multiple of 32", cq.mx_quantize, x.double(), "mxfp4")
    _refused("contiguous", cq.mx_quantize, torch.zeros((64, 64), dtype=torch.bfloat16).t(), "mxfp4")
    _refused("contiguous", cq.mx_quantize, torch.zeros((2, 4, 128), dtype=torch.bfloat16)[:, :, :64], "mxfp4")
    _refused("GPU", cq.mx_quantize, x)
    _refused("GPU", cq.mx_dequantize, codes, scales)
    _refused("scales", cq.mx_dequantize, codes, scales, "mxfp8")
    _refused("uint8", cq.mx_dequantize, codes.view(torch.float8_e4m3fn), scales, "mxfp4")
    _refused("uint8", cq.mx_dequantize, codes.int(), scales)
    _refused("scales", cq.mx_dequantize, codes, scales.int())
    _refused("out_dtype", cq.mx_dequantize, codes, scales, out_dtype=torch.float64)
    k, slots = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    c, e = torch.zeros((5, 2, 16, 64), dtype=torch.uint8), torch.zeros((5, 2, 16, 2), dtype=torch.uint8)
    _refused("bfloat16 or float16", cq.kv_cache_write_mx, k.float(), k.float(), c, e, c, e, slots)
    _refused("bfloat16 or float16", cq.kv_cache_write_mx, k, k[:2], c, e, c, e, slots)
    _refused("int32", cq.kv_cache_write_mx, k, k, c, e, c, e, slots.long())
    _refused("slots", cq.kv_cache_write_mx, k, k, c, e, c, e, slots[:2])
    _refused("contiguous", cq.kv_cache_write_mx, k.transpose(1, 2).contiguous().transpose(1, 2), k, c, e, c, e, slots)
    _refused("GPU", cq.kv_cache_write_mx, k, k, c, e, c, e, slots)


def _linear(ws=None, ws_bytes=0, **kw):
    a = dict(x=FAKE, x_scales=None, qweight=FAKE, scales=FAKE, bias=None, residual=None, y=FAKE, ldx=256, ldxs=0, ldr=0,
             ldy=8, M=4, out=8, inp=256, type=cq.BF16, x_format=cq.MXFP8, y_type=cq.BF16, activation=0, gated=0)
    a.update(kw)
    return cq.load().cq_mxfp4_linear(cq.Mxfp4LinearArgs(**a), ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(type=2), dict(type=-1), dict(y_type=cq.F16), dict(y_type=3), dict(activation=-1), dict(activation=5),
    dict(gated=2), dict(x_format=2), dict(x_format=5), dict(M=-1), dict(out=-1), dict(inp=0), dict(inp=160),
    dict(inp=-128), dict(inp=(1 << 22) + 128, ldx=1 << 23), dict(x_scales=FAKE, ldxs=8, ldx=(1 << 23) + 16), dict(M=1 << 31),
    dict(out=(1 << 25) + 1), dict(out=(1 << 24) + 1, gated=1), dict(inp=1 << 25),
    dict(M=1 << 20, out=1 << 18), dict(M=1 << 19, inp=1 << 15, ldx=1 << 15), dict(x=None), dict(qweight=None), dict(scales=None), dict(y=None), dict(ldx=128),
    dict(ldx=260), dict(ldy=7), dict(residual=FAKE, ldr=7), dict(x=FAKE + 8), dict(qweight=FAKE + 8),
    dict(bias=FAKE + 1), dict(residual=FAKE + 1, ldr=8), dict(y=FAKE + 1), dict(y=FAKE + 2, y_type=cq.F32),
    dict(x_scales=FAKE, ldxs=7), dict(x_scales=FAKE, ldxs=10), dict(x_scales=FAKE + 2, ldxs=8), dict(scales=FAKE + 1),
    dict(x_scales=FAKE, ldxs=8, ldx=255), dict(x_scales=FAKE, ldxs=8, ldx=264),
    dict(x_scales=FAKE, ldxs=8, ldx=112, x_format=cq.MXFP4),
])
def test_linear_rejects_before_launch(kw):
    assert _linear(**kw) == -1


def test_linear_without_rows_or_columns_is_a_no_op():
    assert cq.load().cq_mxfp4_linear(None, None, 0, None) == -1
    assert _linear(M=0, x=None, y=None) == 0 and _linear(out=0, qweight=None) == 0


def test_linear_workspace():
    size = cq.cq_mxfp4_linear_workspace_size
    assert size(8192, 4096, 4096, 0, cq.MXFP4, 1) == 0 and size(1, 4096, 4096, 0, cq.MXFP8, 0) == 0
    for form, each in ((cq.MXFP4, 0.5), (cq.MXFP8, 1.0)):
        need = size(8192, 4096, 4096, 0, form, 0)
        assert 8192 * 4096 * (each + 1 / 32) <= need <= 8192 * 4096 * (each + 1 / 32) + 4096
        assert _linear(M=8192, out=4096, inp=4096, ldx=4096, ldy=4096, x_format=form) == -2
        assert _linear(FAKE, need - 1, M=8192, out=4096, inp=4096, ldx=4096, ldy=4096, x_format=form) == -2
        assert _linear(FAKE + 16, need, M=8192, out=4096, inp=4096, ldx=4096, ldy=4096, x_format=form) == -2
    for bad in ((-1, 8, 128, 0, 3, 0), (4, -8, 128, 0, 3, 0), (4, 8, 100, 0, 3, 0), (4, 8, 128, 2, 3, 0), (4, 8, 128, 0, 0, 0)):
        assert size(*bad) == 0


def test_linear_helper_refuses():
    x, w, s = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((6, 64), dtype=torch.uint8), \
        torch.zeros((6, 4), dtype=torch.uint8)
    _refused("format", cq.mxfp4_linear, x, w, s, x_format="e4m3")
    _refused("matrix", cq.mxfp4_linear, x[0], w, s)
    _refused("bfloat16 or float16", cq.mxfp4_linear, x.float(), w, s)
    _refused("qweight", cq.mxfp4_linear, x, w.int(), s)
    _refused("qweight", cq.mxfp4_linear, x[:, :64], w, s)
    _refused("scales", cq.mxfp4_linear, x, w, s[:, :2])
    _refused("scales", cq.mxfp4_linear, x, w, s.to(torch.bfloat16))
    _refused("even", cq.mxfp4_linear, x, w[:5], s[:5], gated=True)
    _refused("bias", cq.mxfp4_linear, x, w, s, bias=torch.zeros(6))
    _refused("residual", cq.mxfp4_linear, x, w, s, residual=torch.zeros((2, 6)))
    _refused("activation", cq.mxfp4_linear, x, w, s, activation="tanh")
    _refused("contiguous", cq.mxfp4_linear, x, torch.zeros((64, 6), dtype=torch.uint8).t(), s)
    _refused("GPU", cq.mxfp4_linear, x, w, s)
    codes, xs = torch.zeros((2, 128), dtype=torch.uint8), torch.zeros((2, 4), dtype=torch.uint8)
    _refused("scales of x", cq.mxfp4_linear, codes, w, s, x_scales=xs, x_format="mxfp4")
    _refused("uint8", cq.mxfp4_linear, x, w, s, x_scales=xs)
    _refused("residual", cq.mxfp4_linear, codes, w, s, x_scales=xs, bias=torch.zeros(6).half(),
             residual=torch.zeros((2, 6)).bfloat16())


def _attention(ws=None, ws_bytes=0, **kw):
    a = dict(q=FAKE, k_cache=None, v_cache=None, block_table=FAKE, cu_q=FAKE, kv_len=FAKE, out=FAKE, lse=None,
             q_token_stride=256, q_head_stride=64, out_token_stride=256, out_head_stride=64, page_stride=0,
             head_stride=0, row_stride=0, table_stride=4, type=cq.BF16, n_tokens=3, n_requests=2, max_q=2, max_kv=64,
             heads=4, kv_heads=2, head_dim=64, page_size=16, n_pages=9, max_pages=4, causal=1, window=0, scale=0.125)
    cache = _cache(**kw.pop("mx", {}))
    a.update(kw)
    return cq.load().cq_paged_attention_mx(cq.PagedAttentionArgs(**a), cache, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(mx=m) for m in BAD_CACHES] + [
    dict(mx=dict(n_pages=8)), dict(mx=dict(kv_heads=4)), dict(mx=dict(page_size=8)), dict(mx=dict(head_dim=128)),
    dict(mx=dict(k_codes=None)), dict(mx=dict(v_codes=None)), dict(mx=dict(k_scales=None)), dict(mx=dict(v_scales=None)),
    dict(type=cq.F32), dict(n_tokens=-1), dict(n_requests=65536), dict(max_q=-1), dict(heads=3), dict(table_stride=3),
    dict(max_pages=1 << 28, table_stride=1 << 28), dict(causal=2), dict(window=3, causal=0), dict(scale=float("nan")),
    dict(q_token_stride=-256), dict(q_head_stride=60), dict(q=None), dict(out=None), dict(cu_q=None), dict(kv_len=None),
    dict(block_table=None), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(cu_q=FAKE + 1),
])
def test_attention_rejects_before_launch(kw):
    assert _attention(**kw) == -1


def test_attention_workspace_and_limits():
    assert cq.load().cq_paged_attention_mx(None, _cache(), None, 0, None) == -1
    assert cq.load().cq_paged_attention_mx(cq.PagedAttentionArgs(), None, None, 0, None) == -1
    assert _attention(n_tokens=0, q=None) == 0
    assert _attention(max_kv=4096, max_pages=256, table_stride=256) == -2
    assert _attention(ws=FAKE, ws_bytes=1 << 50, n_requests=65535, heads=256, kv_heads=256, max_q=17,
                      mx=dict(kv_heads=256)) == -4


def test_attention_helper_refuses():
    q, t = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4), dtype=torch.int32)
    cu, kv = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c, e = torch.zeros((9, 2, 16, 64), dtype=torch.uint8), torch.zeros((9, 2, 16, 2), dtype=torch.uint8)
    _refused("bfloat16 or float16", cq.paged_attention_mx, q.float(), c, e, c, e, t, cu, kv, 2, 64)
    _refused("int32", cq.paged_attention_mx, q, c, e, c, e, t.long(), cu, kv, 2, 64)
    _refused("cu_q", cq.paged_attention_mx, q, c, e, c, e, t, cu[:2], kv, 2, 64)
    _refused("lse", cq.paged_attention_mx, q, c, e, c, e, t, cu, kv, 2, 64, lse=torch.zeros(3, 4).half())
    _refused("k_cache", cq.paged_attention_mx, q, c[0], e, c, e, t, cu, kv, 2, 64)
    _refused("GPU", cq.paged_attention_mx, q, c, e, c, e, t, cu, kv, 2, 64)
    _refused("k_cache and v_cache", cq._mx_cache, c, e, c[:8], e, 2, 64, -1)
    _refused("strided alike", cq._mx_cache, c, e, c.transpose(1, 2).contiguous().transpose(1, 2), e, 2, 64, -1)
    _refused("mxfp8", cq._mx_cache, c, e, c, e, 2, 256, -1)
    _refused("multiple of 32", cq._mx_cache, c[..., :48], e, c[..., :48], e, 2, 48, -1)
    _refused("k_scales", cq._mx_cache, c, e[..., :1], c, e, 2, 64, -1)
    _refused("k_scales", cq._mx_cache, c, e, c, e[:, :, :8], 2, 64, -1)
    _refused("uint8", cq._mx_cache, c.view(torch.int8), e, c, e, 2, 64, -1)
    _refused("contiguous", cq._mx_cache, *[torch.zeros((9, 2, 64, 16), dtype=torch.uint8).transpose(2, 3), e] * 2, 2, 64, -1)


def test_attention_in_parts_goes_by_what_a_wave_takes():
    """Where a wave would take more tiles of 32 keys than in parts, by one at 256 dimensions and by two at 192, up to 768 keys
    are divided (a workspace is asked for); with fewer dimensions, fewer keys or many requests they are not."""
    size = cq.cq_paged_attention_mx_workspace_size
    for kv in (130, 256):
        assert all(size(1, 1, 1, kv, 32, 8, D) == 0 for D in (32, 64, 96, 128, 160, 192, 224, 256))
    for kv in (257, 512):
        assert all(size(1, 1, 1, kv, 32, 8, D) == 0 for D in (64, 128, 192)) and size(1, 1, 1, kv, 32, 8, 256) > 0
    assert size(1, 1, 1, 768, 32, 8, 128) == 0 and size(1, 1, 1, 768, 32, 8, 160) > 0 and size(1, 1, 1, 768, 32, 8, 256) > 0
    assert all(size(16, 16, 1, 768, 32, 8, D) == 0 for D in (64, 128, 192, 256))
    assert size(1, 1, 1, 769, 32, 8, 64) > 0 and size(1, 1, 1, (1 << 31) - 1, 32, 8, 64) > 0


def test_linear_quantizes_before_where_columns_are_many():
    """5 to 16 rows of values as MXFP8 through more than 16,384 columns are quantized once, into the workspace, not by every tile
    of columns; fewer rows or columns, and MXFP4, are not."""
    size = cq.cq_mxfp4_linear_workspace_size
    for M in (5, 16):
        assert size(M, 16385, 4096, 0, cq.MXFP8, 0) >= M * 4096 * 33 // 32 and size(M, 8193, 4096, 1, cq.MXFP8, 0) > 0
        assert size(M, 16384, 4096, 0, cq.MXFP8, 0) == 0 and size(M, 8192, 4096, 1, cq.MXFP8, 0) == 0
        assert size(M, 128256, 4096, 0, cq.MXFP4, 0) == 0 and size(M, 128256, 4096, 0, cq.MXFP8, 1) == 0
    assert size(4, 128256, 4096, 0, cq.MXFP8, 0) == 0 and size(1, 128256, 4096, 0, cq.MXFP8, 0) == 0
