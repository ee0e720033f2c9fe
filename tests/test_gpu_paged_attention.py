"""GPU: attention over the paged cache (cq_paged_attention) against its definition in 64 bits, within the bound
that oracle.serving.paged_attention derives for each output.  Every slot that no request holds is NaN."""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_amd as cq
from parity import say
from serving import Paged, TORCH, close, i32, t16

pytestmark = pytest.mark.gpu


def _say(*a):
    say("attention:", *a)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hkv,D,page", [(8, 2, 128, 16), (4, 4, 64, 16), (5, 1, 80, 24), (16, 2, 256, 64),
                                          (2, 1, 8, 1), (32, 1, 96, 8), (6, 2, 200, 128)])
def test_single_tokens(H, Hkv, D, page, kind):
    _say("tokens", H, Hkv, D, page, kind)
    Paged([(1, 1), (1, 2), (1, 17), (1, 64), (1, 65), (1, 300)], H, Hkv, D, page, kind).check(cq)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lens", [[(1, 1)], [(5, 5), (3, 40), (1, 9)], [(33, 33), (0, 20), (64, 130)], [(130, 200)],
                                  [(257, 300), (2, 2)]])
@pytest.mark.parametrize("H,Hkv,D,page", [(8, 2, 128, 16), (3, 3, 64, 8), (2, 1, 256, 48)])
def test_chunks(lens, H, Hkv, D, page, kind):
    _say("chunks", lens, H, Hkv, D, page, kind)
    Paged(lens, H, Hkv, D, page, kind, seed=len(lens)).check(cq)


@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 96, 120, 128, 136, 160, 192, 248, 256])
def test_head_dims(D):
    _say("head dim", D)
    Paged([(40, 70), (1, 90)], 4, 2, D, 16, "bf16", seed=D).check(cq)
    Paged([(1, 70), (1, 90)], 4, 2, D, 16, "f16", seed=D).check(cq)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 17, 33])
def test_head_groups(group):
    _say("group", group)
    Paged([(20, 50), (1, 33)], 2 * group, 2, 64, 16, "bf16", seed=group).check(cq)
    Paged([(1, 50), (1, 33)], 2 * group, 2, 64, 16, "bf16", seed=group).check(cq)


@pytest.mark.parametrize("page", [1, 3, 16, 31, 32, 33, 100, 512])
def test_pages_that_end_inside_a_tile(page):
    _say("page", page)
    Paged([(1, 129), (1, 31)], 4, 1, 64, page, "bf16", seed=page).check(cq)
    Paged([(70, 129), (1, 31)], 4, 1, 64, page, "bf16", seed=page).check(cq)


@pytest.mark.parametrize("window", [1, 2, 16, 50, 1000])
@pytest.mark.parametrize("lens", [[(1, 200), (1, 3)], [(90, 200), (7, 7)]])
def test_window(lens, window):
    _say("window", window, lens)
    Paged(lens, 4, 2, 128, 16, "f16", seed=window).check(cq, window=window)


@pytest.mark.parametrize("lens", [[(1, 200)], [(9, 20), (40, 70)], [(150, 150)]])
def test_not_causal(lens):
    _say("not causal", lens)
    Paged(lens, 4, 2, 64, 16, "bf16").check(cq, causal=False)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
def test_scales(scale):
    _say("scale", scale)
    Paged([(1, 90), (50, 60)], 4, 2, 64, 16, "bf16", seed=3).check(cq, scale=scale)
    Paged([(1, 90), (1, 60)], 4, 2, 64, 16, "bf16", seed=3).check(cq, scale=scale)


@pytest.mark.parametrize("lens", [[(1, 5000), (1, 1)], [(1, 20000)], [(3, 4097), (2, 600)], [(100, 2500), (1, 4000)]])
def test_longer_caches(lens):
    _say("longer", lens)
    Paged(lens, 2, 1, 64, 16, "bf16", seed=len(lens)).check(cq)


@pytest.mark.parametrize("lens", [[(4, 4), (1, 1)], [(1, 1), (1, 3)], [(200, 200)]])
def test_rows_that_see_nothing(lens):
    """Fewer cached tokens than new ones, none at all, and tokens that belong to no request."""
    p = Paged(lens, 4, 2, 64, 16, "bf16")
    for kv in ([n - 1 for n, _ in lens], [0] * len(lens), [n // 2 for n, _ in lens]):
        _say("empty", lens, kv)
        p.kv_np = np.array(kv)
        p.kv = i32(kv)
        p.check(cq)
        p.check(cq, causal=True, window=2)
    p.cu_np = np.minimum(p.cu_np, 1)
    p.cu = i32(p.cu_np)
    p.check(cq)


def test_no_requests_and_no_tokens():
    p = Paged([(3, 5)], 2, 1, 64, 16, "f16")
    lse = torch.zeros((3, 2), device="cuda")
    out = p.run(cq, cu_q=i32([0]), kv_len=i32([]), block_table=p.table[:0], lse=lse)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert p.run(cq, q=p.q[:0], cu_q=i32([0, 0])).shape == (0, 2, 64)


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 2, 1 << 30])
@pytest.mark.parametrize("lens,kv", [([(8, 8), (1, 5)], [3, 5]), ([(200, 200)], [150]), ([(300, 300), (2, 9)], [40, 9])])
def test_windows_without_an_end(lens, kv, window):
    """The largest windows equal none, also where the first new tokens stand before position 0."""
    _say("no end", lens, kv, window)
    p = Paged(lens, 4, 2, 64, 16, "bf16", seed=len(lens))
    p.kv_np, p.kv = np.array(kv), i32(kv)
    p.check(cq, window=window)
    assert torch.equal(p.run(cq, window=window), p.run(cq))


@pytest.mark.parametrize("lens", [[(3, 60), (1, 9)], [(70, 90), (2, 9)]])
@pytest.mark.parametrize("window", [0, 20])
def test_lengths_past_the_table_are_those_of_the_table(lens, window):
    """Positions go by the length cut to the table's room: with several new tokens or a window it shows."""
    p = Paged(lens, 4, 2, 64, 8, "bf16")
    room = p.table_np.shape[1] * 8
    for c, t in ((p.kc_np, p.kc), (p.vc_np, p.vc)):          # the request sees the whole last page
        t.copy_(torch.nan_to_num(t, nan=0.5))
        c[np.isnan(c)] = 0.5
    p.kv_np[0] = room
    for past in (1, 1000, (1 << 31) - 1 - room):
        p.kv = i32([room + past, 9])
        p.check(cq, window=window)
    p.kv, p.kv_np[1] = i32([room + 1, -5]), 0
    p.check(cq, window=window)


def _padded(lens, T, front, H, Hkv, D, kind="bf16"):
    """The requests' tokens from number `front` on among T; the others' queries are NaN."""
    p = Paged(lens, H, Hkv, D, 16, kind, seed=T)
    n = p.q.shape[0]
    q, q_np = torch.full((T, H, D), float("nan"), dtype=p.q.dtype, device="cuda"), np.zeros((T, H, D))
    q[front:front + n], q_np[front:front + n] = p.q, p.q_np
    p.q, p.q_np, p.cu_np = q, q_np, p.cu_np + front
    p.cu = i32(p.cu_np)
    return p


@pytest.mark.parametrize("lens", [[(1, 40), (1, 70)], [(40, 60)], [(90, 100), (1, 500), (0, 3)], [(70, 5000)]])
@pytest.mark.parametrize("T,front", [(200, 0), (700, 37), (3001, 0), (9000, 4000)])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (5, 1, 80), (3, 3, 256)])
def test_tokens_of_no_request(lens, T, front, H, Hkv, D):
    """A step padded to a fixed number of tokens: zeros and -inf in front of the requests' tokens and behind them."""
    _say("padded", lens, T, front, H, Hkv, D)
    p = _padded(lens, T, front, H, Hkv, D)
    wide = torch.full((T, H, D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    p.check(cq, out=wide[:, :, :D])
    assert (wide[:, :, D:] == 3).all()


@pytest.mark.parametrize("lens", [[(40, 3000), (1, 2000), (90, 2500)], [(90, 700)] * 3 + [(0, 40)], [(300, 900), (20, 30)]])
@pytest.mark.parametrize("T", [640, 6000])
def test_parts_and_row_tiles_of_a_padded_step(lens, T):
    """Row tiles numbered by the tokens in front of a request and by request, with parts of the keys and without."""
    _say("padded parts", lens, T)
    _padded(lens, T, 0, 8, 2, 64).check(cq)
    _padded(lens, T, 100, 4, 4, 128, "f16").check(cq)


@pytest.mark.parametrize("n,max_q", [(300, 100), (100, 3), (9, 8)])
def test_tokens_past_the_bound_are_left(n, max_q):
    p = Paged([(n, n + 20), (2, 9)], 4, 2, 64, 16, "bf16")
    want, _, tol, _ = p.want()
    out = torch.full_like(p.q, 3.0)
    p.run(cq, max_q=max_q, out=out)
    torch.cuda.synchronize()
    rows = [*range(max_q), n, n + 1]
    close(out[rows], want[rows], tol[rows])
    assert (out[max_q:n] == 3).all()


def _least_us(run, calls=10):
    run()
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(calls):
            run()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1000 / calls)
    return min(times)


@pytest.mark.parametrize("lens", [[(1, 40), (1, 70)], [(33, 60)]])
def test_tokens_of_no_request_cost_their_bytes(lens):
    """They are zeroed by the whole grid: with 8,192 tokens the call takes a few times its own work and a fill of out
    (by a workgroup per key/value head it took 50 times that)."""
    p = _padded(lens, 8192, 0, 32, 8, 128)
    own = p.q[: sum(n for n, _ in lens)].contiguous()
    need = max(256, cq.cq_paged_attention_workspace_size(8192, len(lens), p.max_q, p.max_kv, 32, 8, 128))
    out, ws = torch.empty_like(p.q), torch.empty(need, dtype=torch.uint8, device="cuda")
    padded = _least_us(lambda: p.run(cq, out=out, workspace=ws))
    alone, fill = _least_us(lambda: p.run(cq, q=own, out=out[: own.shape[0]], workspace=ws)), _least_us(out.zero_)
    _say(f"padded {padded:.1f} us, alone {alone:.1f}, fill {fill:.1f}")
    assert padded < 8 * (alone + fill)


@pytest.mark.parametrize("lens", [[(1, 40), (1, 70)], [(50, 80), (3, 9)]])
def test_pages_that_are_not_there(lens):
    """Entries outside the pool count as masked, and kv_len past the table's columns is cut there."""
    p = Paged(lens, 4, 2, 64, 8, "bf16")
    p.table_np[0, 1], p.table_np[0, 3], p.table_np[1, 0] = -1, 1 << 30, p.kc.shape[0]
    p.table = i32(p.table_np)
    p.check(cq)
    p = Paged(lens, 4, 2, 64, 8, "bf16")
    room = p.table_np.shape[1] * 8
    r = int(np.argmax(p.kv_np))
    p.kv = i32([room + 1000 if i == r else k for i, k in enumerate(p.kv_np)])
    for c, t in ((p.kc_np, p.kc), (p.vc_np, p.vc)):          # the row now sees the whole last page
        t.copy_(torch.nan_to_num(t, nan=0.5))
        c[np.isnan(c)] = 0.5
    p.kv_np[r] = room
    p.check(cq)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 3e38])
@pytest.mark.parametrize("lens,first", [([(40, 60)], 50), ([(150, 150)], 64), ([(6, 30)], 27), ([(3, 4)], 2)])
def test_what_later_tokens_hold_does_not_reach_earlier_rows(lens, first, bad):
    """Keys and values from position `first` on are not finite: rows before it keep their values."""
    _say("masked", bad, lens, first)
    for which in ("k", "v", "kv"):
        p = Paged(lens, 4, 2, 64, 16, "bf16", seed=first)
        want, _, tol, _ = p.want()
        pos = np.arange(first, lens[0][1])
        for name, c in (("k", p.kc), ("v", p.vc)):
            if name in which:
                c[p.table[0, pos // 16].long(), :, torch.from_numpy(pos % 16).cuda()] = bad
        out = p.run(cq)
        torch.cuda.synchronize()
        n, kv = lens[0]
        clean = first - (kv - n)
        assert clean > 0
        close(out[:clean], want[:clean], tol[:clean], which)
        if "v" in which and bad != 3e38 and "k" not in which:
            got = out[clean:].float()
            assert (torch.isnan(got) if np.isnan(bad) else got == bad).all()


@pytest.mark.parametrize("lens,window", [([(40, 60)], 8), ([(1, 60)], 8), ([(150, 200)], 70)])
def test_what_left_the_window_does_not_reach_later_rows(lens, window):
    p = Paged(lens, 4, 2, 64, 16, "f16", seed=window)
    want, _, tol, _ = p.want(window=window)
    n, kv = lens[0]
    last = (kv - n) + n // 2 - 1 if n > 1 else kv - window - 1  # positions up to here are NaN
    pos = np.arange(0, last + 1)
    for c in (p.kc, p.vc):
        c[p.table[0, pos // 16].long(), :, torch.from_numpy(pos % 16).cuda()] = float("nan")
    out = p.run(cq, window=window)
    torch.cuda.synchronize()
    rows = [i for i in range(n) if kv - n + i - window >= last]
    assert rows
    close(out[rows], want[rows], tol[rows])


def test_infinite_and_nan_values_that_are_seen():
    """An infinite value spreads as an infinity, both signs or a NaN as NaN, to the rows that see it."""
    p = Paged([(60, 60)], 2, 1, 64, 16, "bf16")
    for (pos, d, v) in ((10, 0, np.inf), (20, 0, -np.inf), (30, 1, np.nan), (5, 2, -np.inf)):
        p.vc[p.table[0, pos // 16].long(), :, pos % 16, d] = v
    out = p.run(cq).float()
    torch.cuda.synchronize()
    assert torch.isfinite(out[:10, :, 0]).all() and (out[10:20, :, 0] == np.inf).all() and torch.isnan(out[20:, :, 0]).all()
    assert torch.isfinite(out[:30, :, 1]).all() and torch.isnan(out[30:, :, 1]).all()
    assert (out[5:, :, 2] == -np.inf).all() and torch.isfinite(out[:, :, 3:]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("lens", [[(60, 60)], [(4, 45)], [(1, 3001)], [(100, 2990)], [(150, 1000), (1, 777)]])
def test_infinities_and_nans_at_every_head_dimension(lens, D, kind):
    """Few rows and many, the keys in one part and in several: an infinite value or a NaN reaches the rows that see it,
    in its own dimension, and nothing else."""
    _say("special", lens, D, kind)
    p = Paged(lens, 2, 1, D, 16, kind, seed=D)
    want, _, tol, _ = p.want()
    n, kv = lens[0]
    seen = np.zeros(want.shape, np.int64)  # 1: an infinity, 2: its negative, 3: both or a NaN
    pos = np.arange(kv - n, kv)[:, None]
    for at, d, what in ((kv - 1 - n // 2, 0, 1), (kv - 1, D - 1, 2), (kv - 1 - n // 3, D // 2 + 1, 3), (kv // 2, 5, 2),
                        (kv // 3, 5, 2), (kv - 1 - n // 4, 7, 1), (kv // 2 + 3, 7, 2), (0, D - 3, 1), (kv - 1, D - 6, 3)):
        p.vc[p.table[0, at // 16].long(), :, at % 16, d] = (np.inf, -np.inf, np.nan)[what - 1]
        seen[:n, :, d] |= np.where(pos >= at, what, 0)
    out = p.run(cq).double().cpu().numpy()
    assert (np.abs(out - want) <= tol)[seen == 0].all()
    assert (out[seen == 1] == np.inf).all() and (out[seen == 2] == -np.inf).all() and np.isnan(out[seen == 3]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(4, 45)], [(60, 60)], [(100, 2990)]])
def test_nans_seen_with_a_weight_of_nothing(lens, D):
    """A key whose weight underflows is seen all the same: 0 times a NaN or an infinity is not a number."""
    _say("weight 0", lens, D)
    p = Paged(lens, 2, 1, D, 16, "bf16", seed=D)
    n, kv = lens[0]
    p.q.fill_(1.0)
    at = kv - 1 - n // 2                                  # seen from the middle row on, its score 400 below the others
    p.kc[p.table[0, at // 16].long(), :, at % 16] = -400.0 * D ** -0.5
    p.vc[p.table[0, at // 16].long(), :, at % 16, :8] = float("nan")
    p.vc[p.table[0, at // 16].long(), :, at % 16, 8:16] = float("inf")
    out = p.run(cq)
    torch.cuda.synchronize()
    first = at - (kv - n)
    assert torch.isfinite(out[:first]).all() and torch.isfinite(out[..., 16:]).all()
    assert torch.isnan(out[first:, :, :8]).all() and not torch.isfinite(out[first:, :, 8:16]).any()


@pytest.mark.parametrize("R", [66, 150])
def test_many_requests_of_every_kind(R):
    """More requests than one search step covers: none, one, few and many new tokens in turn."""
    rng = np.random.default_rng(R)
    lens = []
    for r in range(R):
        n = [1, 90, 0, 20, 130, 65][r % 6]
        lens.append((n, n + int(rng.integers(0, 40))))
    _say("requests", R)
    Paged(lens, 2, 1, 64, 16, "bf16", seed=R).check(cq)
    Paged(lens, 2, 2, 128, 16, "f16", seed=R).check(cq, window=37)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("lens,window", [([(1, 9000), (2, 70)], 0), ([(1, 6000)], 3000), ([(70, 3000)], 0),
                                         ([(90, 2600), (1, 5)], 700)])
def test_parts_of_the_keys(lens, window, D):
    """Few rows against many keys: divided over workgroups and joined, with pages that are not there and a NaN
    behind the last key and in front of the window."""
    _say("parts", lens, window, D)
    p = Paged(lens, 4, 2, D, 16, "bf16" if D % 128 else "f16", seed=D)
    p.table_np[0, 3], p.table_np[0, 90], p.table_np[0, 91] = -1, p.kc.shape[0], -7
    p.table = i32(p.table_np)
    p.check(cq, window=window)


@pytest.mark.parametrize("step", [0.004, 0.03, 0.3, -0.03])
@pytest.mark.parametrize("lens", [[(1, 700)], [(100, 700)]])
@pytest.mark.parametrize("D", [64, 256])
def test_scores_that_climb(D, lens, step):
    """The maximum moves with every key, by steps below and above what the outputs are rescaled for."""
    _say("climb", D, lens, step)
    p = Paged(lens, 2, 1, D, 16, "f16", seed=D)
    p.q, p.q_np = t16(np.ones(p.q.shape), "f16")
    pos = np.arange(lens[0][1])
    rows = (step * pos * D ** -0.5).astype(np.float16).astype(np.float64)
    page, at = p.table_np[0, pos // 16], pos % 16
    for i, x in enumerate(rows):
        p.kc_np[page[i], 0, at[i]] = x
    p.kc.copy_(torch.from_numpy(p.kc_np).half())
    p.check(cq)


@pytest.mark.parametrize("lens", [[(1, 90), (1, 50)], [(70, 90), (2, 50)]])
def test_strides_and_orders(lens):
    """q out of packed q-k-v rows, out into wider rows, the cache token-major, the table wider than needed."""
    p = Paged(lens, 6, 2, 64, 16, "f16", order="nhd", table_extra=5)
    T = p.q.shape[0]
    wide = torch.zeros((T, 10, 64), dtype=torch.float16, device="cuda")
    wide[:, 2:8] = p.q
    dest = torch.full((T, 6, 80), 3.0, dtype=torch.float16, device="cuda")
    bt = torch.full((len(lens), p.table.shape[1] + 3), 1 << 29, dtype=torch.int32, device="cuda")
    bt[:, : p.table.shape[1]] = p.table
    p.check(cq, q=wide[:, 2:8], out=dest[:, :, 8:72], block_table=bt[:, : p.table.shape[1]])
    assert (dest[:, :, :8] == 3).all() and (dest[:, :, 72:] == 3).all()


def test_one_allocation_for_both_caches_and_heads_outside():
    """K and V interleaved per page: [pages, 2, kv_heads, page, D]."""
    p = Paged([(1, 60), (30, 40)], 4, 2, 64, 16, "bf16")
    both = torch.stack((p.kc, p.vc), dim=1)
    p.check(cq, k_cache=both[:, 0], v_cache=both[:, 1])


@pytest.mark.parametrize("lens", [[(1, 700)], [(100, 300)]])
def test_bounds_larger_and_smaller_than_the_lengths(lens):
    """max_q and max_kv only divide the work: larger bounds, and a kv_len beyond max_kv, change nothing but the
    order of sums."""
    p = Paged(lens, 4, 2, 64, 16, "bf16")
    p.check(cq, max_q=lens[0][0] + 300, max_kv=20000)
    p.check(cq, max_kv=16)


@pytest.mark.parametrize("lens", [[(1, 3000), (1, 100)], [(200, 500), (1, 900)]])
def test_same_bits_again_and_on_another_stream(lens):
    p = Paged(lens, 8, 2, 128, 16, "bf16")
    a = p.run(cq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = p.run(cq, stream=s)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(a, p.run(cq))


@pytest.mark.parametrize("lens", [[(1, 3000), (1, 100)], [(100, 200), (1, 900)]])
def test_replayed_graph(lens):
    p = Paged(lens, 8, 2, 64, 16, "f16")
    T, H, D = p.q.shape
    need = cq.cq_paged_attention_workspace_size(T, len(lens), p.max_q, p.max_kv, H, 2, D)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(p.q)
    p.run(cq, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run(cq, out=out, workspace=ws)
    for k in range(4):
        p.q.copy_(torch.randn_like(p.q))
        p.kv.copy_(i32([max(1, kv - 7 * k) for _, kv in lens]))
        eager = p.run(cq)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k


def test_cache_past_32_bit_offsets():
    """The requests' pages lie past 2^31 elements of a cache of 4 GiB and more."""
    p = Paged([(1, 40), (20, 30)], 4, 2, 128, 16, "bf16")
    far = (1 << 31) // (2 * 16 * 128) + 1
    n = p.kc.shape[0]
    big = [torch.empty((far + n, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    big[0][far:], big[1][far:] = p.kc, p.vc
    p.check(cq, k_cache=big[0], v_cache=big[1], block_table=torch.where(p.table >= 0, p.table + far, p.table))


def test_the_new_tokens_own_keys_through_the_other_operators():
    """Block map, cache write and attention in turn: prompts in two chunks, then tokens one by one, against the
    whole prompts at once."""
    H, Hkv, D, page, n = 4, 2, 64, 16, [50, 33, 7]
    torch.manual_seed(0)
    q, k, v = (torch.randn((sum(n), h, D), device="cuda").half() for h in (H, Hkv, Hkv))
    start = np.concatenate([[0], np.cumsum(n)])
    kc, vc = (torch.full((40, Hkv, page, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    free, left = torch.randperm(40, device="cuda").int(), i32([40])
    ctx, got = i32([0, 0, 0]), torch.zeros_like(q)
    for step in ([20, 33, 1], [29, 0, 5], [1, 0, 1]):
        m = cq.kv_block_map(ctx, i32(step), free, left, table, page, sum(step) + 2)
        at = np.concatenate([start[r] + int(c) + np.arange(s) for r, (c, s) in enumerate(zip(ctx.tolist(), step))])
        at = torch.from_numpy(at).cuda()
        pad = torch.cat([at, at[:2]])                          # two padding tokens, slot -1
        cq.kv_cache_write(k[pad], v[pad], kc, vc, m["slots"])
        got[at] = cq.paged_attention(q[at], kc, vc, table, m["cu_q"], m["kv_len"], max(step), 64)
        ctx, left = m["kv_len"], m["n_left"]
    torch.cuda.synchronize()
    assert ctx.tolist() == n and left.tolist() == [40 - 4 - 3 - 1]
    qd, kd, vd = (t.double().cpu() for t in (q, k, v))
    for r in range(3):
        a, b = start[r], start[r + 1]
        for h in range(H):
            s = qd[a:b, h] @ kd[a:b, h // 2].T * D ** -0.5
            s = s.masked_fill(torch.ones_like(s).triu(1).bool(), -np.inf)
            want = torch.softmax(s, -1) @ vd[a:b, h // 2]
            w = torch.softmax(s, -1) @ vd[a:b, h // 2].abs()
            # weights and output rounded to f16, scores within 2^-16 of exact at these sizes
            assert ((got[a:b, h].double().cpu() - want).abs() <= (2.0 ** -11 + 2.0 ** -14) * w + 2.0 ** -11 * want.abs() + 2.0 ** -24).all()


def test_refusals():
    p = Paged([(1, 20)], 4, 2, 64, 16, "bf16")
    for kw in (dict(q=p.q.half()), dict(q=p.q[..., :32]), dict(k_cache=p.kc.float()), dict(v_cache=p.vc[:2]),
               dict(cu_q=p.cu.long()), dict(kv_len=i32([1, 2])), dict(block_table=p.table[0]),
               dict(lse=torch.zeros((1, 3), device="cuda")), dict(out=torch.zeros((1, 4, 64), device="cuda")),
               dict(q=p.q.cpu()), dict(q=p.q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            p.run(cq, **kw)
    for kw in (dict(q=torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda")), dict(window=-1),
               dict(window=4, causal=False), dict(scale=float("inf")), dict(scale=float("nan")), dict(max_q=-1),
               dict(q=torch.zeros((3, 4, 68), dtype=torch.bfloat16, device="cuda")[..., :64])):
        with pytest.raises(cq.CQError):
            p.run(cq, **kw)
    odd = Paged([(1, 20)], 2, 1, 8, 16, "bf16")
    with pytest.raises(cq.CQError):                            # head_dim 4
        odd.run(cq, q=odd.q[..., :4].contiguous(), k_cache=odd.kc[..., :4].contiguous(),
                v_cache=odd.vc[..., :4].contiguous())
