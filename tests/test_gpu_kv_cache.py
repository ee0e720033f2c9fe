"""GPU: block tables and slot maps (cq_kv_block_map) and cache writes (cq_kv_cache_write): whole numbers and
copies, equal to the definition's."""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_amd as cq
from oracle import serving as ref
from parity import say
from serving import TORCH, i32

pytestmark = pytest.mark.gpu


def _check(ctx, new, page, most, free, n_free=None, max_tokens=None, pad=0, seed=0):
    rng = np.random.default_rng(seed)
    R = len(ctx)
    n_free = len(free) if n_free is None else n_free
    max_tokens = int(np.clip(new, 0, None).sum()) if max_tokens is None else max_tokens
    table = np.full((R, most), -1, np.int64)
    for r in range(R):
        have = max(0, min(most, -(-int(ctx[r]) // page)))
        table[r, :have] = rng.integers(0, 1000, have) + 5000
    want = ref.block_map(ctx, new, free, n_free, table, page, max_tokens)
    buf = torch.full((R, most + pad), -7, dtype=torch.int32, device="cuda")
    bt = buf[:, :most]
    bt.copy_(i32(table))
    got = cq.kv_block_map(i32(ctx), i32(new), i32(free), i32([n_free]), bt, page, max_tokens)
    torch.cuda.synchronize()
    for k, v in dict(got, block_table=bt).items():
        assert np.array_equal(v.cpu().numpy().astype(np.int64), want[k]), k
    assert (buf[:, most:] == -7).all()
    return want


@pytest.mark.parametrize("page", [1, 7, 8, 16, 24, 128])
@pytest.mark.parametrize("R", [1, 2, 63, 64, 65, 300])
def test_lengths(R, page):
    say(f"block map: R={R} page={page}")
    rng = np.random.default_rng(R * page)
    ctx, new = rng.integers(0, 200, R), rng.integers(0, 40, R)
    _check(ctx, new, page, 240 // page + 2, rng.permutation(R * 60 + 10), pad=R % 3)


@pytest.mark.parametrize("R", [1000, 1025, 2500, 4096])
def test_many_requests(R):
    rng = np.random.default_rng(R)
    _check(rng.integers(0, 500, R), rng.integers(0, 6, R), 16, 40, rng.permutation(R * 2), max_tokens=R * 6)


def test_exact_page_borders_and_empty_requests():
    _check([0, 16, 15, 31, 0, 32, 47], [0, 16, 1, 1, 1, 0, 2], 16, 4, np.arange(20)[::-1].copy())


def test_pool_runs_out():
    w = _check([0, 3, 8, 0], [8, 1, 9, 4], 4, 8, np.arange(4), max_tokens=64)
    assert list(w["status"]) == [0, 0, 1, 1]


def test_no_pages_and_bad_counts():
    w = _check([3, 4], [1, 0], 4, 4, np.arange(3), n_free=0)
    assert list(w["status"]) == [0, 0]
    _check([3, 4], [2, 0], 4, 4, np.arange(3), n_free=-5)
    _check([3, 4], [2, 9], 4, 4, np.arange(3), n_free=100)


def test_token_buffer_runs_out():
    w = _check([0, 0, 0], [5, 5, 5], 4, 4, np.arange(40), max_tokens=12)
    assert list(w["status"]) == [0, 0, 1]
    _check([0, 0], [5, 0], 4, 4, np.arange(40), max_tokens=0)


def test_invalid_lengths_take_nothing():
    w = _check([-1, 2, 0, 60, 5], [4, -3, 6, 10, 2147483647], 4, 16, np.arange(40), max_tokens=40)
    assert list(w["status"]) == [2, 2, 0, 2, 2]


def test_refused_then_invalid():
    w = _check([0, 0, -4, 1], [4, 400, 1, 1], 4, 128, np.arange(9), max_tokens=500)
    assert list(w["status"]) == [0, 1, 2, 1]


def test_one_long_prompt():
    rng = np.random.default_rng(5)
    _check([100, 7], [70001, 1], 16, 5000, rng.permutation(4400), max_tokens=70010)


@pytest.mark.parametrize("R", [5, 70, 1100])
def test_sums_past_32_bits(R):
    """Lengths whose sums pass 2^32, behind requests that fit."""
    new = [1 << 20, 0] + [1 << 30] * (R - 3) + [1]
    _check([0] * R, new, 1 << 20, 2047, np.arange(1000), max_tokens=(1 << 20) + 5)
    _check([(1 << 30) - 1] * R, [1] * R, 1 << 20, 2047, np.arange(50), max_tokens=60)


def test_no_requests():
    got = cq.kv_block_map(i32([]), i32([]), i32([1, 2]), i32([2]), torch.zeros((0, 3), dtype=torch.int32, device="cuda"),
                          16, 5)
    torch.cuda.synchronize()
    assert got["cu_q"].tolist() == [0] and got["n_left"].tolist() == [2] and got["slots"].tolist() == [-1] * 5


def test_slots_beyond_32_bits_and_pages_missing():
    """A page whose slot would pass 2^31 - 1, and a held page entered as -1, give -1."""
    bt = i32([[-1, 3], [5, -1]])
    got = cq.kv_block_map(i32([10, 16]), i32([1, 2]), i32([1 << 30]), i32([1]), bt, 16, 3)
    torch.cuda.synchronize()
    assert got["slots"].tolist() == [-1, -1, -1] and bt.tolist() == [[-1, 3], [5, 1 << 30]]


def test_block_map_refusals():
    one, t = i32([1]), i32([[1, 2]])
    ok = dict(ctx_len=one, new_len=one, free_pages=one, n_free=one.clone(), block_table=t, page_size=4, max_tokens=3)
    for kw in (dict(new_len=i32([1, 2])), dict(ctx_len=one.long()), dict(n_free=i32([1, 2])), dict(block_table=i32([1])),
               dict(block_table=i32([[1, 2], [3, 4]]).t()[:1]), dict(free_pages=one.cpu())):
        with pytest.raises(ValueError):
            cq.kv_block_map(**dict(ok, **kw))
    for kw in (dict(page_size=0), dict(page_size=1 << 30)):
        with pytest.raises(cq.CQError):
            cq.kv_block_map(**dict(ok, **kw))
    many = torch.zeros(cq.MAX_REQUESTS + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(cq.CQError):
        cq.kv_block_map(many, many, one, i32([1]), many[:, None], 16, 3)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,D,page,order", [(1, 1, 8, 1, "hnd"), (5, 2, 128, 16, "hnd"), (33, 3, 80, 24, "nhd"),
                                              (300, 8, 64, 16, "nhd"), (7, 2, 12, 8, "hnd"), (9, 2, 7, 8, "hnd"),
                                              (2000, 4, 128, 64, "hnd")])
def test_cache_write(T, H, D, page, order, kind):
    say(f"cache write: T={T} H={H} D={D} page={page} {order} {kind}")
    g = torch.Generator().manual_seed(T)
    n_pages = T // page + 5
    qkv = torch.randn((T, 3, H, D), generator=g).to(TORCH[kind]).cuda()
    k, v = qkv[:, 1], qkv[:, 2]
    shape = (n_pages, H, page, D) if order == "hnd" else (n_pages, page, H, D)
    caches = [torch.randn(shape, generator=g).to(TORCH[kind]).cuda() for _ in range(2)]
    if order == "nhd":
        caches = [c.transpose(1, 2) for c in caches]
    want = [c.clone() for c in caches]
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[::5] = torch.tensor([-1, n_pages * page, -(1 << 31), 2147483647], dtype=torch.int32).repeat(T)[: slots[::5].numel()]
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < n_pages * page:
            want[0][s // page, :, s % page] = k[t]
            want[1][s // page, :, s % page] = v[t]
    cq.kv_cache_write(k, v, caches[0], caches[1], slots.cuda())
    torch.cuda.synchronize()
    assert torch.equal(caches[0], want[0]) and torch.equal(caches[1], want[1])


def test_cache_write_past_32_bit_offsets():
    """A cache of 2^32 bytes and more each: the last page lies past 2^31 elements."""
    page, H, D = 256, 16, 256
    n_pages = (1 << 31) // (page * H * D) + 3
    kc = torch.empty((n_pages, H, page, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    k, v = (torch.randn((2, H, D), device="cuda").bfloat16() for _ in range(2))
    cq.kv_cache_write(k, v, kc, vc, i32([n_pages * page - 1, 3]))
    torch.cuda.synchronize()
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[0, :, 3], v[1]) and torch.equal(vc[-1, :, -1], v[0])


def test_cache_write_refusals():
    c = torch.zeros((2, 1, 4, 8), dtype=torch.float16, device="cuda")
    k, s = torch.zeros((3, 1, 8), dtype=torch.float16, device="cuda"), i32([0, 1, 2])
    for kw in (dict(k=k[:2]), dict(v=k.bfloat16()), dict(slots=s.long()), dict(v_cache=c[:1]), dict(k_cache=c.float()),
               dict(k=k.transpose(0, 2).contiguous().transpose(0, 2)), dict(v_cache=c.transpose(1, 2).contiguous().transpose(1, 2)[:, :, :, :4]),
               dict(slots=s.cpu())):
        with pytest.raises(ValueError):
            cq.kv_cache_write(**dict(dict(k=k, v=k, k_cache=c, v_cache=c.clone(), slots=s), **kw))
    cq.kv_cache_write(k[:0], k[:0], c, c, s[:0])
