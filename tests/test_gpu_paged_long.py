"""Paged attention where a CTA works through many key tiles and several items
one after another: rings that wrap, queries and outputs handed over, maxima
that move on in late tiles, waits that run out far into a share.  The plan,
compiled for the host, says what a CTA has to do in each case."""
import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from tests import paged_plan
from tests.helpers import check_status, status_word
from tests.paged_cases import FP16_TINY, TYPES, attention_bounds, values
from tests.test_gpu_paged import SENTINEL, same_bits
from tests.test_gpu_paged_values import mma_sum_loss

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


# ------------------------------------------------------------------ growing maxima
def climbing(seed, n, lens, Hq, H, D, dtype, ps, step):
    """Sequences of n[b] tokens over lens[b] rows whose keys have a component
    along one direction that grows by `step` (of a logit, for a temperature of 1)
    from 128 rows to the next, as every query has one: the maximum of a row
    under a positive temperature keeps moving on, under a negative one it is
    among the first keys.  Page i of every sequence is one of three."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-max(lens) // ps)
    u = torch.full((D,), D ** -0.5, device="cuda")
    rows = torch.arange(width * ps, device="cuda").view(width, 1, 1, ps, 1)
    k = torch.randn(width, 3, H, ps, D, generator=g, device="cuda") * 0.4
    k += u * (rows * (step / 128 / 4.0 * D ** 0.5))                     # q's component: 4
    v = torch.randn(width, 3, H, ps, D, generator=g, device="cuda")
    q = torch.randn(sum(n), Hq, D, generator=g, device="cuda") * 0.4 + 4.0 * u
    rng = np.random.default_rng(seed)
    pick = np.arange(width)[None] * 3 + rng.integers(0, 3, (len(n), width))
    t = TYPES[dtype]
    d = {"q": q.to(t), "k_pages": k.view(-1, H, ps, D).to(t), "v_pages": v.view(-1, H, ps, D).to(t),
         "page_table": torch.from_numpy(pick.astype(np.int32)).cuda(),
         "cache_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "cu_tokens": torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")}
    size = vark.vark_paged_attention_workspace(sum(n), len(n), Hq, H, D, ps, width)
    d["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return d


def reference(d, n, lens, tau, causal, missed=0):
    """In 64 bits: outputs, log-sums, the weighted mean of |v| and the largest sum
    of |q k| (see oracle.paged.paged_attention).  A planted mistake: the first
    `missed` keys weigh 2^8 too much, as if one step of the maximum had not
    reached their sum."""
    q, kp, vp = (d[x].double() for x in ("q", "k_pages", "v_pages"))
    N, Hq, D = q.shape
    H = kp.shape[1]
    G = Hq // H
    out, mean_abs = torch.zeros_like(q), torch.zeros_like(q)
    lse, logit_abs = (torch.zeros(N, Hq, dtype=torch.float64, device="cuda") for _ in range(2))
    f = torch.from_numpy(tau).cuda().double() * D ** -0.5
    at = 0
    for b in range(len(n)):
        ids = d["page_table"][b].long()
        for h in range(H):
            K, V = (x[ids, h].reshape(-1, D)[:lens[b]] for x in (kp, vp))
            rows, heads = slice(at, at + n[b]), slice(h * G, (h + 1) * G)
            Q = q[rows, heads]
            x = torch.einsum("ngd,kd->ngk", Q, K) * f[heads, None]
            big = torch.einsum("ngd,kd->ngk", Q.abs(), K.abs()) * f[heads, None].abs()
            if causal:
                unseen = (torch.arange(lens[b], device="cuda")[None] >
                          torch.arange(n[b], device="cuda")[:, None] + lens[b] - n[b])[:, None]
                x, big = x.masked_fill(unseen, -torch.inf), big.masked_fill(unseen, 0.0)
            x[..., :missed] += 8 * np.log(2.0)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[..., None])
            out[rows, heads], mean_abs[rows, heads] = p @ V, p @ V.abs()
            lse[rows, heads], logit_abs[rows, heads] = z, big.amax(-1)
        at += n[b]
    return [t.cpu().numpy() for t in (out, lse, mean_abs, logit_abs)]


CLIMBS = [
    # rows of an item, tokens, rows of the caches, G, H, page, causal, step of the maximum
    (16, 1, (1000, 3000), 4, 4, 16, True, 3.0),
    (16, 3, (900, 2500), 5, 4, 64, True, 6.0),
    (32, 1, (1000, 3000), 20, 4, 32, True, 3.0),
    (32, 5, (1200, 2600), 6, 4, 256, False, 4.0),
    (256, 100, (1000, 3000), 4, 4, 128, True, 3.0),
    (256, 33, (1100, 2800), 8, 4, 16, False, 7.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", range(len(CLIMBS)))
def test_many_items_whose_maxima_climb(case, D, dtype):
    R, tokens, (lo, hi), G, H, ps, causal, step = CLIMBS[case]
    rng = np.random.default_rng(case)
    B = 80 if R == 256 else 180
    n = [tokens] * B
    lens = [int(x) for x in rng.integers(lo, hi, B)]
    segments, _, _, whole, _ = paged_plan.plan(R, n, lens, H, G, causal)
    per_cta = np.bincount(segments[:, 0])
    long = np.bincount(segments[:, 0], weights=segments[:, 5] - segments[:, 4] >= 6)
    assert not whole and (per_cta >= 3).mean() > 0.9 and (long >= 2).mean() > 0.9
    d = climbing(case, n, lens, G * H, H, D, dtype, ps, step)
    tau = np.resize(np.array([1.0, 1.5, -0.5, 0.0, 0.3, -1.5], dtype=np.float32), G * H)
    out, lse = attend(d, causal, torch.from_numpy(tau).cuda())
    check_against(d, n, lens, tau, causal, out, lse, dtype, R == 256)


def check_against(d, n, lens, tau, causal, out, lse, dtype, tiles):
    D = d["q"].shape[-1]
    o, z, mean_abs, logit_abs = reference(d, n, lens, tau, causal)
    keys = float(max(lens))
    b_out, b_lse = attention_bounds(o, z, mean_abs, logit_abs, keys, dtype, D)
    if dtype == "fp16":
        # a probability is off by FP16_TINY of 2^7 at most, not of 1; |v| is at most 6
        b_out += 6.0 * keys * FP16_TINY * (2.0 ** -7 - 1.0)
    b_out += mma_sum_loss(keys, tiles) * mean_abs
    bad = ~(np.abs(values(out) - o) <= b_out)
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(values(out) - o)[bad].max())
    assert (np.abs(lse.cpu().double().numpy() - z) <= b_lse).all()
    # the bound is one that a step of the maximum, missed once, would pass
    planted, *_ = reference(d, n, lens, tau, causal, missed=512)
    assert (np.abs(planted - o) > b_out).any(axis=(0, 2))[tau > 0].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_sums_taken_out_of_the_accumulators_while_maxima_climb(D, dtype):
    """Segments of more than 256 and 512 key tiles on tcgen05, the maximum moving
    on between."""
    n, lens = [70] * 126, [40000 + 9000 * b for b in range(14)] * 9
    G, H, ps = 4, 1, 256
    segments, *_ = paged_plan.plan(256, n, lens, H, G, True)
    runs = segments[:, 5] - segments[:, 4]
    assert (runs > 256).sum() > 50 and (runs > 512).sum() > 20
    d = climbing(3, n, lens, G * H, H, D, dtype, ps, 0.1)
    tau = np.array([1.0, 0.2, -0.5, 0.0], dtype=np.float32)
    out, lse = attend(d, True, torch.from_numpy(tau).cuda())
    check_against(d, n, lens, tau, True, out, lse, dtype, True)
