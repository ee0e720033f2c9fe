"""Inputs and comparisons shared by the GPU tests of the serving operators."""
import numpy as np
import torch

from oracle import serving as ref

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def t16(a, kind):
    """A device tensor of the 16-bit type, and the float64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[kind])
    return t.to("cuda"), t.double().numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to("cuda")


def close(got, want, tol, label=""):
    got = got.detach().double().cpu().numpy()
    err = np.abs(got - want)
    assert got.shape == want.shape
    assert np.all(err <= tol), f"{label}: error {err.max():.3g}, {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"


class Paged:
    """Requests (new tokens, cached tokens with them) over a shuffled pool of pages.  What no request holds of
    the pool is NaN."""

    def __init__(self, lens, H, Hkv, D, page, kind, seed=0, spare=3, order="hnd", table_extra=0):
        rng = np.random.default_rng(seed)
        self.kind, self.lens, self.page = kind, lens, page
        pages = [-(-kv // page) for _, kv in lens]
        n_pages = sum(pages) + spare
        perm = rng.permutation(n_pages)
        self.table_np = np.full((len(lens), max(pages + [1]) + table_extra), -1)
        at = 0
        kc, vc = (np.full((n_pages, Hkv, page, D), np.nan, np.float32) for _ in range(2))
        for r, ((_, kv), p) in enumerate(zip(lens, pages)):
            self.table_np[r, :p] = perm[at:at + p]
            at += p
            for b in range(p):
                m = min(page, kv - b * page)
                for c in (kc, vc):
                    c[self.table_np[r, b], :, :m] = rng.standard_normal((Hkv, m, D))
        self.cu_np = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int64)
        self.kv_np = np.array([kv for _, kv in lens], np.int64)
        T = int(self.cu_np[-1])
        self.q, self.q_np = t16(rng.standard_normal((T, H, D)), kind)
        self.kc, self.kc_np = t16(kc, kind)
        self.vc, self.vc_np = t16(vc, kind)
        if order == "nhd":
            self.kc, self.vc = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (self.kc, self.vc))
        self.table, self.cu, self.kv = i32(self.table_np), i32(self.cu_np), i32(self.kv_np)
        self.max_q, self.max_kv = max([n for n, _ in lens] + [0]), max([k for _, k in lens] + [0])
        self.scale = D ** -0.5

    def run(self, cq, **kw):
        kw = dict(dict(q=self.q, k_cache=self.kc, v_cache=self.vc, block_table=self.table, cu_q=self.cu,
                       kv_len=self.kv, max_q=self.max_q, max_kv=self.max_kv), **kw)
        return cq.paged_attention(**kw)

    def want(self, causal=True, window=0, scale=None):
        return ref.paged_attention(self.q_np, self.kc_np, self.vc_np, self.table_np, self.cu_np, self.kv_np,
                                   self.scale if scale is None else scale, causal, window, self.kind)

    def check(self, cq, causal=True, window=0, scale=None, **kw):
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        out = self.run(cq, causal=causal, window=window, scale=scale, lse=lse, **kw)
        torch.cuda.synchronize()
        want, wl, tol, ltol = self.want(causal, window, scale)
        close(out, want, tol, "out")
        got = lse.double().cpu().numpy()
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(got), empty)
        assert np.all(np.abs(got[~empty] - wl[~empty]) <= ltol[~empty]), "lse"
        return out
