"""The serving operators' C entry points without a GPU: bad arguments are refused before anything reaches HIP."""
import pytest
import torch

import post_weight_quantization_group_amd as cq

FAKE = 1 << 20  # a 16-byte-aligned address that is never dereferenced: every call below fails its checks


def _linear(**kw):
    a = dict(x=FAKE, ldx=256, xt=cq.BF16, qw=FAKE, sc=FAKE, bias=None, res=None, ldr=0, act=0, gated=0, M=4, out=8,
             inp=256, y=FAKE, ldy=8, yt=cq.BF16)
    a.update(kw)
    return cq.load().cq_w4a16_linear(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(xt=2), dict(xt=-1), dict(yt=cq.F16), dict(yt=3), dict(act=-1), dict(act=5), dict(gated=2), dict(M=-1),
    dict(out=-1), dict(inp=0), dict(inp=130), dict(inp=-128), dict(M=1 << 31), dict(out=1 << 31),
    dict(out=1 << 30, gated=1), dict(inp=1 << 25), dict(x=None), dict(qw=None), dict(sc=None), dict(y=None),
    dict(ldx=128), dict(ldx=260), dict(ldy=7), dict(res=FAKE, ldr=7), dict(x=FAKE + 8), dict(qw=FAKE + 2),
    dict(sc=FAKE + 1), dict(bias=FAKE + 1), dict(res=FAKE + 1, ldr=8), dict(y=FAKE + 1), dict(y=FAKE + 2, yt=cq.F32),
])
def test_linear_rejects_before_launch(kw):
    assert _linear(**kw) == -1


def test_linear_without_rows_or_columns_is_a_no_op():
    assert _linear(M=0, x=None, y=None) == 0 and _linear(out=0, qw=None) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int32, torch.int8])
def test_linear_refuses_scales_that_are_not_binary16(dtype):
    """16 bits of another type (bfloat16) would be read as binary16."""
    x, qw = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((16, 8), dtype=torch.int32)
    with pytest.raises(ValueError, match="scales"):
        cq.w4a16_linear(x, qw, torch.zeros((1, 8), dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.float16, torch.int16, torch.uint16])
def test_linear_takes_scales_as_binary16_or_its_bits(dtype):
    """They pass the check of their type: what is refused on the CPU is where the arrays live."""
    x, qw = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((16, 8), dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        cq.w4a16_linear(x, qw, torch.zeros((1, 8), dtype=dtype))


def _map(**kw):
    a = dict(ctx=FAKE, new=FAKE + 64, R=2, page=16, free=FAKE + 128, n_free=FAKE + 192, cap=4, table=FAKE + 256,
             stride=3, most=3, tokens=5, cu=FAKE + 512, kv=FAKE + 640, slots=FAKE + 704, pos=FAKE + 768,
             status=FAKE + 832, left=FAKE + 896)
    a.update(kw)
    return cq.load().cq_kv_block_map(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(R=-1), dict(R=cq.MAX_REQUESTS + 1), dict(page=0), dict(most=0), dict(most=1 << 27, stride=1 << 27),
    dict(stride=2), dict(tokens=-1), dict(cap=-1), dict(free=None), dict(n_free=None), dict(left=None),
    dict(left=FAKE + 192), dict(cu=None), dict(ctx=None), dict(new=None), dict(table=None), dict(kv=None),
    dict(status=None), dict(slots=None), dict(pos=None), dict(kv=FAKE), dict(kv=FAKE + 64), dict(status=FAKE),
    dict(slots=FAKE + 706), dict(table=FAKE + 258),
])
def test_block_map_rejects_before_launch(kw):
    assert _map(**kw) == -1


def _write(**kw):
    a = dict(k=FAKE, kt=16, kh=8, v=FAKE, vt=16, vh=8, kc=FAKE, vc=FAKE, ps=64, hs=32, rs=8, pages=4, page=4, heads=2,
             D=8, slots=FAKE, T=3)
    a.update(kw)
    return cq.load().cq_kv_cache_write(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(pages=-1), dict(heads=0), dict(page=0), dict(D=0), dict(kt=-1), dict(vh=-8), dict(ps=-64),
    dict(rs=-1), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(slots=None), dict(k=FAKE + 1),
    dict(vc=FAKE + 1), dict(slots=FAKE + 2),
])
def test_cache_write_rejects_before_launch(kw):
    assert _write(**kw) == -1


def test_cache_write_of_nothing_is_a_no_op():
    assert _write(T=0, k=None) == 0 and _write(pages=0, kc=None) == 0


def _attention(ws=None, ws_bytes=0, **kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, cu_q=FAKE, kv_len=FAKE, out=FAKE, lse=None,
             q_token_stride=256, q_head_stride=64, out_token_stride=256, out_head_stride=64, page_stride=2048,
             head_stride=1024, row_stride=64, table_stride=4, type=cq.BF16, n_tokens=3, n_requests=2, max_q=2,
             max_kv=64, heads=4, kv_heads=2, head_dim=64, page_size=16, n_pages=9, max_pages=4, causal=1, window=0,
             scale=0.125)
    a.update(kw)
    return cq.load().cq_paged_attention(cq.PagedAttentionArgs(**a), ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(type=cq.F32), dict(n_tokens=-1), dict(n_requests=-1), dict(n_requests=65536), dict(max_q=-1),
    dict(max_kv=-1), dict(kv_heads=0), dict(heads=3), dict(heads=1), dict(heads=1 << 17), dict(head_dim=0),
    dict(head_dim=60), dict(head_dim=264), dict(n_tokens=1 << 30), dict(page_size=0), dict(n_pages=-1),
    dict(max_pages=-1), dict(table_stride=3), dict(max_pages=1 << 28, table_stride=1 << 28), dict(causal=2),
    dict(window=-1), dict(window=3, causal=0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(q_token_stride=-256), dict(q_head_stride=60), dict(row_stride=68), dict(page_stride=4), dict(q=None),
    dict(out=None), dict(cu_q=None), dict(kv_len=None), dict(k_cache=None), dict(v_cache=None),
    dict(block_table=None), dict(q=FAKE + 8), dict(k_cache=FAKE + 2), dict(out=FAKE + 8), dict(lse=FAKE + 2),
    dict(cu_q=FAKE + 1),
])
def test_attention_rejects_before_launch(kw):
    assert _attention(**kw) == -1


def test_attention_workspace():
    assert cq.load().cq_paged_attention(None, None, 0, None) == -1
    assert _attention(n_tokens=0, q=None) == 0
    size = cq.cq_paged_attention_workspace_size
    assert size(-1, 1, 1, 1, 1, 1, 64) == 0 and size(1, 1, 1, 1, 1, 1, 63) == 0 and size(1, 1, 1, 1, 3, 2, 64) == 0


@pytest.mark.parametrize("T,R,max_q,max_kv", [(8192, 1, 32, 8192), (8192, 1, 33, 1 << 20), (16384, 8, 64, 4096),
                                              (1 << 20, 3, 100, 9000), (60, 1, 60, 8192), (8192, 0, 32, 8192)])
@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 128), (8, 1, 256), (16, 16, 64)])
def test_attention_workspace_goes_by_the_rows_that_can_exist(T, R, max_q, max_kv, H, Hkv, D):
    """A step padded to T tokens needs no more than 256 workgroups' rows, D sums and two statistics each."""
    assert cq.cq_paged_attention_workspace_size(T, R, max_q, max_kv, H, Hkv, D) <= 256 * 256 * (D + 2) * 4


@pytest.mark.parametrize("kw", [dict(n_requests=65535, heads=256, kv_heads=256, max_q=17),
                                dict(n_tokens=(1 << 30) - 1, heads=2, kv_heads=2, max_q=(1 << 30) - 1, n_requests=2)])
def test_attention_grid_too_large_is_refused_before_launch(kw):
    """More row tiles than a launch can number: refused by the entry point, not by a launch in the middle of the call."""
    assert _attention(ws=FAKE, ws_bytes=1 << 50, **kw) == -4
