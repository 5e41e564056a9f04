"""Paged attention where a CTA works through many key tiles and several items
one after another: rings that wrap, queries and outputs handed over, waits
that run out far into a share."""
import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from tests.helpers import check_status, status_word
from tests.test_gpu_paged import SENTINEL, same_bits

pytestmark = pytest.mark.gpu


def shared_pages(rng, B, n, keys, Hq, H, D, dtype, ps=64, n_pages=48):
    """B sequences of n tokens over `keys` rows each, out of a small pool whose
    pages all of them read (a table of random pages)."""
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    d = {name: torch.randn(n_pages, H, ps, D, generator=g).to(dtype).cuda() for name in ("k_pages", "v_pages")}
    width = -(-keys // ps)
    d["page_table"] = torch.from_numpy(rng.integers(0, n_pages, (B, width)).astype(np.int32)).cuda()
    d["cache_len"] = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    d["cu_tokens"] = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    d["q"] = torch.randn(B * n, Hq, D, generator=g).to(dtype).cuda()
    size = vark.vark_paged_attention_workspace(B * n, B, Hq, H, D, ps, width)
    d["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return d


def attend(d, causal=True, tau=None, status=None):
    st = status_word() if status is None else status
    out = torch.full_like(d["q"], SENTINEL)
    lse = torch.full(d["q"].shape[:2], SENTINEL, device="cuda")
    vark.vark_paged_attention(d["q"], d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"], tau,
                              causal, out, lse, d["workspace"], st)
    if status is None:
        check_status(st)
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 4), (1, 24), (70, 4)])
@pytest.mark.parametrize("tile", [1, 2, 5, 7, 14])
def test_waits_that_run_out_far_into_a_share(D, n, G, tile, monkeypatch):
    """A key tile that never comes, after the ring has wrapped or in a later
    item: every warp of every kernel gives up, the call reports it, and the next
    one gives what one before gave."""
    rng = np.random.default_rng(D + n + tile)
    d = shared_pages(rng, 60, n, 600, 4 * G, 4, D, torch.bfloat16)         # 240 items of 5 tiles: 8.1 a CTA
    want = attend(d)
    monkeypatch.setenv("VARK_TEST_WAIT_LIMIT_MS", "50")
    monkeypatch.setenv("VARK_TEST_WITHHOLD_KV_TILE", str(tile))
    st = status_word()
    attend(d, status=st)
    torch.cuda.synchronize()
    # (items of 70 x 4 rows are two of 256: 480 of 5 tiles, 16.2 a CTA)
    assert int(st.item()) == (-6 if tile < (16 if n > 1 else 8) else 0)
    monkeypatch.delenv("VARK_TEST_WAIT_LIMIT_MS")
    monkeypatch.delenv("VARK_TEST_WITHHOLD_KV_TILE")
    got = attend(d)
    assert same_bits(got[0], want[0]) and torch.equal(got[1], want[1])
