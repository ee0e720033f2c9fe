"""GPU: the serving helpers make their arrays' GPU current for the call where another one is.  One GPU is enough: the
binding is told that another is current until it has switched."""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_amd as cq
from serving import Paged, close, i32

pytestmark = pytest.mark.gpu


@pytest.fixture
def elsewhere(monkeypatch):
    """The GPUs that calls have switched to."""
    entered, device = [], torch.cuda.device

    class Switch(device):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(cq, "_device_now", lambda: entered[-1] if entered else 7)
    return entered


def test_linear(elsewhere):
    x, out = torch.randn((3, 128), device="cuda").bfloat16(), torch.zeros((3, 8), device="cuda")
    qw = torch.full((16, 8), 0x7FFFFFFF, dtype=torch.int32, device="cuda")  # codes 7, and -1 last of a word
    y = cq.w4a16_linear(x, qw, torch.ones((1, 8), device="cuda").half(), residual=torch.ones((3, 8), device="cuda").bfloat16(),
                        activation="relu", out_dtype=torch.float32, out=out)
    want = (7 * x.double().view(3, 16, 8)[..., :7].sum((1, 2)) - x.double().view(3, 16, 8)[..., 7].sum(1)).clamp(min=0) + 1
    assert elsewhere == [0] and y is out and torch.allclose(y.double(), want[:, None].expand(3, 8), rtol=1e-4, atol=1e-4)


def test_map_and_write(elsewhere):
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    m = cq.kv_block_map(i32([0]), i32([5]), i32([1, 0, 2]), i32([3]), table, 4, 6)
    assert elsewhere == [0] and m["slots"].tolist() == [8, 9, 10, 11, 0, -1] and table.tolist() == [[2, 0, -1, -1]]
    del elsewhere[:]
    k = torch.randn((6, 1, 8), device="cuda").half()
    kc, vc = (torch.zeros((3, 1, 4, 8), dtype=torch.float16, device="cuda") for _ in range(2))
    cq.kv_cache_write(k, -k, kc, vc, m["slots"])
    assert elsewhere == [0] and torch.equal(kc[2, 0], k[:4, 0]) and torch.equal(vc[0, 0, 0], -k[4, 0]) and not kc[1].any()


def test_attention(elsewhere):
    p = Paged([(2, 40), (1, 9)], 4, 2, 64, 16, "bf16")
    out = p.run(cq, window=7, scale=0.2)
    assert elsewhere == [0]
    want, _, tol, _ = p.want(window=7, scale=0.2)
    close(out, want, tol)
