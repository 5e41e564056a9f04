"""Norm and rotation of queries and keys, the append to a paged cache and
attention over it, against the fp64 oracle: element by element, with the
rounding bounds of tests/paged_cases.py; every row no call may touch keeps its
bits."""
import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from oracle import paged as ref
from tests.helpers import check_status, status_word
from tests.paged_cases import (HALF, TYPES, Pages, attention_bounds, norm_bound, rope_table, rounded, values)

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16).cpu(), b.contiguous().view(torch.int16).cpu())


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,norm,weight,rope_dim,pairs", [
    (1, 1, 1, 1, 64, vark.VARK_NORM_RMS, True, 64, False),
    (2, 5, 9, 3, 128, vark.VARK_NORM_RMS, True, 128, False),
    (3, 7, 8, 8, 128, vark.VARK_NORM_L2, False, 128, True),
    (1, 33, 17, 2, 64, vark.VARK_NORM_L2, True, 32, False),
    (2, 3, 5, 1, 128, vark.VARK_NORM_NONE, True, 48, True),
    (1, 2, 4, 4, 128, vark.VARK_NORM_NONE, False, 16, False),
    (2, 9, 3, 2, 64, vark.VARK_NORM_RMS, False, 0, False),
])
def test_norm_rope(dtype, B, T, Hq, Hk, D, norm, weight, rope_dim, pairs):
    rng = np.random.default_rng(B * 100 + T)
    eps = 1e-5
    host = [rounded(rng.standard_normal((B, T, H, D)) * 3, dtype) for H in (Hq, Hk)]
    host[0][0, 0, 0] = 0                       # a row of zeros
    w = [rng.uniform(0.5, 1.5, D).astype(np.float32) if weight else None for _ in range(2)]
    table = rope_table(40, rope_dim) if rope_dim else None
    pos = rng.integers(0, 40, size=(B, T)).astype(np.int32) if rope_dim else None
    if rope_dim and T > 2:
        pos[0, 1] = -1                         # a padding token
    st = status_word()
    dev = [t.cuda() for t in host]
    outs = [torch.full_like(t, SENTINEL) for t in dev]
    wd = [None if x is None else torch.from_numpy(x).cuda() for x in w]
    vark.vark_qk_norm_rope(dev[0], dev[1], outs[0], outs[1], norm, wd[0], wd[1], eps,
                           None if table is None else torch.from_numpy(table).cuda(),
                           None if pos is None else torch.from_numpy(pos).cuda(), st, pairs=pairs)
    check_status(st)
    for x, got, wt in zip(host, outs, w):
        H = x.shape[2]
        p = np.zeros(B * T, dtype=np.int64) if pos is None else pos.reshape(-1)
        y, mag = ref.norm_rotate(values(x).reshape(B * T, H, D), norm, wt, eps, table, p, pairs)
        g = values(got).reshape(B * T, H, D)
        live = p >= 0
        assert (np.abs(g - y) <= norm_bound(y, mag, dtype, D))[live].all()
        assert (g[~live] == SENTINEL).all()


def test_norm_rope_strides_in_place_and_single_tensor():
    """A fused projection's slices in, head-major out; in place; keys only."""
    rng = np.random.default_rng(5)
    B, T, Hq, Hk, D = 2, 11, 6, 2, 128
    qkv = rounded(rng.standard_normal((B, T, Hq + 2 * Hk, D)), "bf16").cuda()
    keep = qkv.clone()
    table = torch.from_numpy(rope_table(64, 64)).cuda()
    pos = torch.arange(B * T, dtype=torch.int32, device="cuda").view(B, T)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    st = status_word()
    plain = [torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())]
    vark.vark_qk_norm_rope(q.contiguous(), k.contiguous(), *plain, vark.VARK_NORM_RMS, None, None, 1e-6, table, pos, st)
    major = [torch.empty(B, H, T, D, dtype=q.dtype, device="cuda").transpose(1, 2) for H in (Hq, Hk)]
    vark.vark_qk_norm_rope(q, k, *major, vark.VARK_NORM_RMS, None, None, 1e-6, table, pos, st)
    for a, b in zip(plain, major):
        assert same_bits(a, b)
    only = torch.empty_like(plain[1])
    vark.vark_qk_norm_rope(None, k, None, only, vark.VARK_NORM_RMS, None, None, 1e-6, table, pos, st)
    assert same_bits(only, plain[1])
    vark.vark_qk_norm_rope(q, k, q, k, vark.VARK_NORM_RMS, None, None, 1e-6, table, pos, st)
    check_status(st)
    assert same_bits(q, plain[0]) and same_bits(k, plain[1])
    assert same_bits(qkv[:, :, Hq + Hk:], keep[:, :, Hq + Hk:])      # the values between are not touched


def test_norm_rope_position_behind_the_table_is_recorded_and_skipped():
    x = torch.ones(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(x, SENTINEL)
    st = status_word()
    pos = torch.tensor([[0, 9, 1]], dtype=torch.int32, device="cuda")
    vark.vark_qk_norm_rope(x, None, o, None, vark.VARK_NORM_L2, None, None, 1e-6,
                           torch.from_numpy(rope_table(9, 64)).cuda(), pos, st)
    torch.cuda.synchronize()
    assert int(st.item()) == -2
    assert (o[0, 1] == SENTINEL).all() and (o[0, 0] != SENTINEL).all() and (o[0, 2] != SENTINEL).all()


# ------------------------------------------------------------------ append
APPENDS = [
    # n, lens (per sequence, or per sequence and head), H, D, page, head_pages, rope_dim, pairs, norm
    ([1], [1], 1, 64, 16, False, 64, False, vark.VARK_NORM_RMS),
    ([3, 0, 40, 1], [3, 5, 57, 16], 2, 128, 16, False, 128, False, vark.VARK_NORM_RMS),
    ([17, 33], [100, 33], 9, 64, 32, False, 32, True, vark.VARK_NORM_L2),
    ([5, 2], [3, 300], 3, 128, 256, False, 0, False, vark.VARK_NORM_NONE),      # a cache shorter than its chunk
    ([4, 9], [[4, 20, 9], [9, 100, 130]], 3, 128, 64, True, 128, False, vark.VARK_NORM_L2),
    ([1] * 70, list(range(1, 71)), 4, 64, 16, False, 64, False, vark.VARK_NORM_RMS),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_paged_append(dtype, case):
    n, lens, H, D, page, head, rope_dim, pairs, norm = APPENDS[case]
    rng = np.random.default_rng(case)
    pg = Pages(rng, dtype, n, lens, H, D, page, head)
    pad, eps = 3, 1e-6
    N = int(pg.cu[-1]) + pad
    # strided sources: k and v as slices of one tensor
    kv = rounded(rng.standard_normal((N, 2 * H + 1, D)) * 2, dtype)
    k, v = kv[:, :H], kv[:, H:2 * H]
    w = rng.uniform(0.5, 1.5, D).astype(np.float32)
    table = rope_table(50, rope_dim) if rope_dim else None
    pos = rng.integers(0, 50, size=N).astype(np.int32)
    if N > 8:
        pos[1] = -1                                     # not stored
    d = pg.cuda()
    st = status_word()
    kvd = kv.cuda()
    vark.vark_paged_append(kvd[:, :H], kvd[:, H:2 * H], d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                           d["cache_len"], norm, torch.from_numpy(w).cuda(), eps,
                           None if table is None else torch.from_numpy(table).cuda(),
                           torch.from_numpy(pos).cuda() if rope_dim else None, st, pairs=pairs)
    check_status(st)
    y, mag = ref.norm_rotate(values(k), norm, w, eps, table, pos, pairs)
    bound = norm_bound(y, mag, dtype, D)
    want_k, want_v = pg.k.clone(), pg.v.clone()
    gk, gv = d["k_pages"].cpu(), d["v_pages"].cpu()
    for b in range(len(n)):
        for i in range(n[b]):
            t = int(pg.cu[b]) + i
            if rope_dim and pos[t] < 0:
                continue
            for h in range(H):
                at = ref.paged_row(pg.table, pg.lens, pg.cu, page, b, h, i)
                if at is None:
                    continue
                idx = at if head else (at[0], h, at[1])
                assert (np.abs(values(gk[idx]) - y[t, h]) <= bound[t, h]).all(), (b, i, h)
                want_k[idx] = gk[idx]
                want_v[idx] = v[t, h]
    assert same_bits(gv, want_v)
    assert same_bits(gk, want_k)                         # every other row kept its bits


def test_paged_append_bad_tables_are_recorded_and_skipped():
    rng = np.random.default_rng(0)
    pg = Pages(rng, "bf16", [4, 4], [20, 20], 2, 64, 16, False)
    k = rounded(rng.standard_normal((8, 2, 64)), "bf16").cuda()
    for what, value in (("page_table", 10 ** 6), ("page_table", -1), ("cache_len", 10 ** 6)):
        d = pg.cuda()
        if what == "page_table":
            d[what][0, 1] = value
        else:
            d[what][0] = value
        before = d["k_pages"].clone()
        st = status_word()
        vark.vark_paged_append(k, k, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                               vark.VARK_NORM_NONE, None, 0.0, None, None, st)
        torch.cuda.synchronize()
        assert int(st.item()) == -2
        page = int(pg.table[1, 1])                       # the second sequence is stored all the same
        assert same_bits(d["k_pages"][page, :, 0:4].transpose(0, 1), k[4:8])
        d["k_pages"][page] = before[page]
        assert same_bits(d["k_pages"], before)


# ------------------------------------------------------------------ attention
ATTENTION = [
    # n, lens, Hq, H, D, page, head_pages, causal
    ([1], [1], 1, 1, 64, 16, False, True),
    ([1], [777], 8, 2, 128, 16, False, True),
    ([1, 1, 1], [1, 129, 2000], 3, 1, 128, 64, False, True),
    ([1, 0, 1, 1], [16, 40, 17, 0], 4, 4, 64, 32, False, True),          # no token; no key
    ([5, 3], [260, 3], 6, 2, 128, 128, False, True),
    ([5, 3], [260, 3], 6, 2, 128, 256, False, False),
    ([7, 4], [3, 1], 4, 2, 64, 16, False, True),                          # queries that see nothing
    ([40, 1, 130], [300, 90, 130], 4, 2, 128, 16, False, True),
    ([130], [513], 5, 1, 64, 32, False, True),
    ([9, 25], [[9, 100], [300, 25]], 2, 2, 128, 16, True, False),
    ([64], [[64, 70, 900]], 6, 3, 128, 128, True, False),
    ([33], [[33, 160]], 32, 2, 64, 64, True, True),
    ([1] * 40, list(range(3, 43)), 16, 1, 128, 16, False, True),
    ([260], [260], 2, 1, 128, 64, False, True),
    ([300, 7], [1000, 600], 3, 1, 128, 128, False, False),
    ([5, 9, 12], [200, 9, 70], 4, 2, 64, 16, False, True),
    ([6, 3, 0, 7], [500, 90, 5, 40], 16, 4, 128, 256, False, False),
    ([9, 8], [[700, 9], [5, 33]], 4, 2, 64, 32, True, True),
    ([200, 200], [200, 1500], 4, 4, 64, 16, False, True),
]


def run_attention(pg, q, tau, causal, extra_tokens=0, stream=None):
    d = pg.cuda()
    N, Hq, D = q.shape
    out = torch.full((N, Hq, D), SENTINEL, dtype=q.dtype, device="cuda")
    lse = torch.full((N, Hq), SENTINEL, dtype=torch.float32, device="cuda")
    ws = torch.empty(vark.vark_paged_attention_workspace(N, len(pg.cu) - 1, Hq, pg.H, D, pg.page,
                                                         pg.table.shape[-1]), dtype=torch.uint8, device="cuda")
    st = status_word()
    vark.vark_paged_attention(q.cuda(), d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                              None if tau is None else torch.from_numpy(tau).cuda(), causal, out, lse, ws, st)
    check_status(st)
    return out, lse


def compare(pg, q, tau, causal, out, lse, dtype):
    N, Hq, D = q.shape
    t = np.ones(Hq, dtype=np.float32) if tau is None else tau
    o, z, mean_abs, logit_abs = ref.paged_attention(values(q), pg.cu, values(pg.k), values(pg.v), pg.table, pg.lens, t,
                                                    causal)
    keys = float(max(1, pg.lens.max(initial=1)))
    b_out, b_lse = attention_bounds(o, z, mean_abs, logit_abs, keys, dtype, D)
    live = int(pg.cu[-1])
    g, gz = values(out), lse.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(g - o) <= b_out)[:live]
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(g - o)[:live][bad].max())
    dead = np.isneginf(z)[:live]
    assert (np.isneginf(gz[:live]) == dead).all()
    assert (np.abs(np.where(dead, 0, gz[:live]) - np.where(dead, 0, z[:live])) <= b_lse[:live])[~dead].all()
    assert (g[live:] == SENTINEL).all() and (gz[live:] == SENTINEL).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_paged_attention(dtype, case):
    n, lens, Hq, H, D, page, head, causal = ATTENTION[case]
    rng = np.random.default_rng(100 + case)
    pg = Pages(rng, dtype, n, lens, H, D, page, head, extra_width=case % 2)
    N = int(pg.cu[-1]) + (case % 3)
    q = rounded(rng.standard_normal((N, Hq, D)), dtype)
    tau = rng.uniform(0.5, 2.0, Hq).astype(np.float32) if case % 4 else None
    out, lse = run_attention(pg, q, tau, causal)
    compare(pg, q, tau, causal, out, lse, dtype)


def test_paged_attention_large_logits():
    """Rows whose maximum jumps in a late tile, and logits of hundreds."""
    rng = np.random.default_rng(3)
    pg = Pages(rng, "bf16", [3], [900], 2, 128, 32, False)
    q = rounded(rng.standard_normal((3, 4, 128)) * 12, "bf16")
    tau = np.array([1.0, 2.0, -1.0, 0.0], dtype=np.float32)       # any sign: also all logits 0
    out, lse = run_attention(pg, q, tau, True)
    compare(pg, q, tau, True, out, lse, "bf16")


def test_paged_attention_is_deterministic_and_takes_strided_queries():
    rng = np.random.default_rng(8)
    for n, lens, Hq, H in (([1, 1, 1], [700, 30, 3000], 8, 2), ([90, 300], [700, 300], 4, 2)):
        pg = Pages(rng, "bf16", n, lens, H, 128, 16, False)
        N = int(pg.cu[-1])
        qkv = rounded(rng.standard_normal((N, Hq + 2 * H, 128)), "bf16").cuda()
        d = pg.cuda()
        ws = torch.empty(vark.vark_paged_attention_workspace(N, len(n), Hq, H, 128, 16, pg.table.shape[-1]),
                         dtype=torch.uint8, device="cuda")
        st = status_word()
        outs = []
        for q in (qkv[:, :Hq], qkv[:, :Hq], qkv[:, :Hq].contiguous()):
            out = torch.empty(Hq, N, 128, dtype=q.dtype, device="cuda").transpose(0, 1)     # head-major
            ws.random_(0, 255)                                  # the workspace holds nothing between calls
            vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                                      None, True, out, None, ws, st)
            outs.append(out)
        check_status(st)
        assert same_bits(outs[0], outs[1]) and same_bits(outs[0], outs[2])


@pytest.mark.parametrize("n", [[1, 1], [150, 20]])
def test_paged_attention_bad_tables_are_recorded(n):
    """Both kernels: pages, lengths and offsets outside the arguments are
    recorded, and a good call on the same context works afterwards."""
    rng = np.random.default_rng(4)
    pg = Pages(rng, "bf16", n, [200, 260], 2, 64, 16, False)
    N = int(pg.cu[-1])
    q = rounded(rng.standard_normal((N, 4, 64)), "bf16")
    ws = torch.empty(vark.vark_paged_attention_workspace(N, 2, 4, 2, 64, 16, pg.table.shape[-1]), dtype=torch.uint8,
                     device="cuda")
    for key, index, value in (("page_table", (0, 3), 10 ** 7), ("page_table", (1, 0), -5), ("cache_len", (1,), 10 ** 7),
                              ("cache_len", (0,), -1), ("cu_tokens", (2,), N + 1), ("cu_tokens", (1,), -3)):
        d = pg.cuda()
        d[key][index] = value
        out, st = torch.empty(N, 4, 64, dtype=torch.bfloat16, device="cuda"), status_word()
        vark.vark_paged_attention(q.cuda(), d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                                  d["cache_len"], None, True, out, None, ws, st)
        torch.cuda.synchronize()
        assert int(st.item()) == -2, (key, index)
    out, lse = run_attention(pg, q, None, True)
    compare(pg, q, None, True, out, lse, "bf16")


@pytest.mark.parametrize("n", [[1, 1], [150, 20]])
def test_withheld_tile_times_out_and_context_stays_usable(n, monkeypatch):
    rng = np.random.default_rng(6)
    pg = Pages(rng, "bf16", n, [3000, 2600], 2, 128, 32, False)
    N = int(pg.cu[-1])
    q = rounded(rng.standard_normal((N, 4, 128)), "bf16")
    d = pg.cuda()
    ws = torch.empty(vark.vark_paged_attention_workspace(N, 2, 4, 2, 128, 32, pg.table.shape[-1]), dtype=torch.uint8,
                     device="cuda")
    monkeypatch.setenv("VARK_TEST_WAIT_LIMIT_MS", "100")
    monkeypatch.setenv("VARK_TEST_WITHHOLD_KV_TILE", "0")
    out, st = torch.empty(N, 4, 128, dtype=torch.bfloat16, device="cuda"), status_word()
    vark.vark_paged_attention(q.cuda(), d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                              None, True, out, None, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == -6
    monkeypatch.delenv("VARK_TEST_WAIT_LIMIT_MS")
    monkeypatch.delenv("VARK_TEST_WITHHOLD_KV_TILE")
    out, lse = run_attention(pg, q, None, True)
    rows = [0, N - 1]
    o, z, mean_abs, logit_abs = ref.paged_attention(values(q), pg.cu, values(pg.k), values(pg.v), pg.table, pg.lens,
                                                    np.ones(4), True)
    b_out, _ = attention_bounds(o, z, mean_abs, logit_abs, 3000.0, "bf16", 128)
    assert (np.abs(values(out) - o) <= b_out)[rows].all()


def test_pages_beyond_32_bit_offsets():
    """Pages that lie past 2^31 elements and past 4 GB of the pool."""
    rng = np.random.default_rng(11)
    H, ps, D = 8, 64, 128
    n_pages = (1 << 31) // (H * ps * D) + 40
    pg = Pages(rng, "bf16", [1, 40], [130, 170], H, D, ps, False)
    N, Hq = int(pg.cu[-1]), 16
    q = rounded(rng.standard_normal((N, Hq, D)), "bf16").cuda()
    kv = rounded(rng.standard_normal((N, H, D)), "bf16").cuda()
    small, st = pg.cuda(), status_word()
    big = dict(small)
    at = n_pages - pg.k.shape[0]
    for name in ("k_pages", "v_pages"):
        big[name] = torch.zeros(n_pages, H, ps, D, dtype=torch.bfloat16, device="cuda")
        big[name][at:] = small[name]
    big["page_table"] = torch.where(small["page_table"] >= 0, small["page_table"] + at, small["page_table"])
    outs = []
    for d in (small, big):
        vark.vark_paged_append(kv, kv, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                               vark.VARK_NORM_L2, None, 1e-6, None, None, st)
        for lo in (0, 1):                       # one token a sequence, then the chunk
            cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda") if lo == 0 else d["cu_tokens"]
            n = 2 if lo == 0 else N
            out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(vark.vark_paged_attention_workspace(n, 2, Hq, H, D, ps, d["page_table"].shape[1]),
                             dtype=torch.uint8, device="cuda")
            vark.vark_paged_attention(q[:n], cu, d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"], None,
                                      True, out, None, ws, st)
            outs.append(out)
    check_status(st)
    assert same_bits(outs[0], outs[2]) and same_bits(outs[1], outs[3])
    assert not torch.isnan(outs[0].float()).any()


# ------------------------------------------------------------------ runs of the calls
def sequence_step(x, d, rope, pos, ws, st, out, q_rot, causal, tau=None):
    """One layer's step: queries turned, keys and values appended, attention."""
    q, k, v = x
    vark.vark_qk_norm_rope(q[None], None, q_rot[None], None, vark.VARK_NORM_RMS, None, None, 1e-6, rope, pos[None], st)
    vark.vark_paged_append(k, v, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                           vark.VARK_NORM_RMS, None, 1e-6, rope, pos, st)
    vark.vark_paged_attention(q_rot, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"], tau,
                              causal, out, None, ws, st)


def test_tokens_one_by_one_equal_a_causal_chunk():
    """A sequence taken token by token, in two chunks and at once gives the same
    cache bit for bit, and outputs within the rounding of two results."""
    rng = np.random.default_rng(21)
    T, Hq, H, D, ps = 77, 8, 2, 128, 16
    x = [rounded(rng.standard_normal((T, h, D)), "bf16").cuda() for h in (Hq, H, H)]
    rope = torch.from_numpy(rope_table(T, D)).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    st = status_word()
    results = []
    for cuts in ([T], [40, T], list(range(1, T + 1))):
        d = dict(k_pages=torch.zeros(8, H, ps, D, dtype=torch.bfloat16, device="cuda"),
                 page_table=torch.tensor([[6, 1, 4, 0, 7]], dtype=torch.int32, device="cuda"))
        d["v_pages"] = torch.zeros_like(d["k_pages"])
        out, q_rot = torch.empty_like(x[0]), torch.empty_like(x[0])
        a = 0
        for z in cuts:
            d["cu_tokens"] = torch.tensor([0, z - a], dtype=torch.int32, device="cuda")
            d["cache_len"] = torch.tensor([z], dtype=torch.int32, device="cuda")
            ws = torch.empty(vark.vark_paged_attention_workspace(z - a, 1, Hq, H, D, ps, 5), dtype=torch.uint8,
                             device="cuda")
            sequence_step([t[a:z] for t in x], d, rope, pos[a:z], ws, st, out[a:z], q_rot[a:z], True)
            a = z
        check_status(st)
        results.append((d["k_pages"], d["v_pages"], values(out)))
    for k, v, out in results[1:]:
        assert same_bits(k, results[0][0]) and same_bits(v, results[0][1])
        # each is off by at most 2 half steps of the type of mean |v| <= 4.5 here, and its own half step
        assert np.abs(out - results[0][2]).max() <= 2 * (2 * HALF["bf16"] * 4.5)


def test_scales_over_head_pages_match_the_pruned_cache():
    """Generation by scales under a head-specific keep schedule: every head's
    retained rows lie in its own pages, past_len of the offset tables giving
    their number, and a dropped scale is overwritten by the next append.  The
    same queries, keys and values through the compacted cache."""
    import synth
    from tests.helpers import Tables
    sides = synth.SIDES_TINY
    S, B, H, D, ps = len(sides), 2, 4, 64, 16
    rng = np.random.default_rng(31)
    keep = rng.integers(0, 2, size=(1, H, S)).astype(np.uint8)
    keep[:, :, 0] = 1
    tab = Tables(keep, sides, B, D)
    rows = int(sum(s * s for s in sides))
    width = -(-rows // ps)
    perm = rng.permutation(B * H * width).astype(np.int32).reshape(B, H, width)
    table = torch.from_numpy(perm).cuda()
    pool = [torch.zeros(B * H * width, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kc, vc = (torch.zeros(max(tab.total, 8), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tau = torch.from_numpy(rng.uniform(0.5, 2, H).astype(np.float32)).cuda()
    st = status_word()
    for k in range(S):
        nk = sides[k] ** 2
        q, kn, vn = (rounded(rng.standard_normal((B, H, nk, D)), "bf16").cuda() for _ in range(3))
        want = torch.empty_like(q)
        vark.vark_pruned_attention_step(q, kc, vc, tab.kc_rows(0), kn, vn, sides, k, tab.head_off[0], tab.seg_off[0],
                                        tab.past_len[0], tau, None, want, st)
        vark.vark_append_scale(kn, vn, B * H * nk * D, 1, B, H, sides, D, k, tab.keep, tab.head_off, tab.seg_off,
                               tab.layer_base, kc, vc)
        tokens = [t.transpose(1, 2).reshape(B * nk, H, D) for t in (q, kn, vn)]
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * nk
        length = (tab.past_len[0, :, k] + nk).expand(B, H).contiguous()
        vark.vark_paged_append(tokens[1], tokens[2], cu, *pool, table, length, vark.VARK_NORM_NONE, None, 0.0, None,
                               None, st)
        got = torch.empty_like(tokens[0])
        ws = torch.empty(vark.vark_paged_attention_workspace(B * nk, B, H, H, D, ps, width), dtype=torch.uint8,
                         device="cuda")
        vark.vark_paged_attention(tokens[0], cu, *pool, table, length, tau, False, got, None, ws, st)
        check_status(st)
        diff = values(got.view(B, nk, H, D).transpose(1, 2)) - values(want)
        # both within half a step of their probabilities and outputs of mean |v| <= 5
        assert np.abs(diff).max() <= 2 * (2 * HALF["bf16"] * 5.0), k


@pytest.mark.parametrize("n", [[1, 1, 1], [60, 130, 3]])
def test_captured_steps_replay_with_new_lengths(n):
    """A captured step reads lengths, tables, positions and values when it is
    replayed; two graphs of one stream share a workspace; calls on two streams
    with a workspace each run at the same time."""
    rng = np.random.default_rng(41)
    H, Hq, D, ps, B = 2, 8, 128, 16, 3
    top = [400, 700, 300]
    pg = Pages(rng, "bf16", n, top, H, D, ps, False)
    N = int(pg.cu[-1])
    rope = torch.from_numpy(rope_table(1024, D)).cuda()
    pos = torch.zeros(N, dtype=torch.int32, device="cuda")
    x = [rounded(rng.standard_normal((N, h, D)), "bf16").cuda() for h in (Hq, H, H)]
    st = status_word()
    size = vark.vark_paged_attention_workspace(N, B, Hq, H, D, ps, pg.table.shape[-1])
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    bufs = [(torch.empty_like(x[0]), torch.empty_like(x[0])) for _ in range(3)]
    d = pg.cuda()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def fill(step):
        r = np.random.default_rng(step)
        for t in x:
            t.copy_(rounded(r.standard_normal(tuple(t.shape)), "bf16"))
        d["cache_len"].copy_(torch.tensor([a - step * 17 for a in top], dtype=torch.int32))
        pos.copy_(torch.from_numpy(r.integers(0, 1024, N).astype(np.int32)))
        torch.cuda.synchronize()

    fill(0)
    graphs = []
    for b in range(2):
        with torch.cuda.stream(streams[0]):
            sequence_step(x, d, rope, pos, ws[0], st, *bufs[b], True)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            sequence_step(x, d, rope, pos, ws[0], st, *bufs[b], True)
        graphs.append(g)
    for step in (1, 2, 5):
        fill(step)
        sequence_step(x, d, rope, pos, ws[1], st, *bufs[2], True)
        torch.cuda.synchronize()
        want = bufs[2][0].clone()
        for b in range(2):
            bufs[b][0].fill_(SENTINEL)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graphs[0].replay()
            graphs[1].replay()
        check_status(st)
        assert same_bits(bufs[0][0], want) and same_bits(bufs[1][0], want)
    # two streams at once (the cache is only read)
    for b in range(2):
        bufs[b][0].fill_(SENTINEL)
    torch.cuda.synchronize()
    for rep in range(20):
        for b, s in enumerate(streams):
            with torch.cuda.stream(s):
                vark.vark_paged_attention(bufs[2][1], d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                                          d["cache_len"], None, True, bufs[b][0], None, ws[b], st)
    check_status(st)
    assert same_bits(bufs[0][0], want) and same_bits(bufs[1][0], want)
    # a stream given by hand
    bufs[0][0].fill_(SENTINEL)
    torch.cuda.synchronize()
    vark.vark_paged_attention(bufs[2][1], d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                              None, True, bufs[0][0], None, ws[0], st, stream=streams[1])
    streams[1].synchronize()
    assert same_bits(bufs[0][0], want)
