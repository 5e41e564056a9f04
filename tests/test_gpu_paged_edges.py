"""The serving calls where a caller may well go and the other tests do not:
many query heads a kv head, pages of 256 rows under long chunks, temperatures
of any sign on every kernel, empty and all-padding chunks, offsets outside the
chunk, pages that sequences share, tables written on the stream just before a
call, and both ways through the binding."""
import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from oracle import paged as ref
from tests.helpers import check_status, status_word
from tests.paged_cases import Pages, attention_bounds, rope_table, rounded, values
from tests.test_gpu_paged import SENTINEL, compare, run_attention, same_bits

pytestmark = pytest.mark.gpu

CASES = [
    # n, lens, Hq, H, D, page, head_pages, causal
    ([1, 1], [300, 40], 40, 1, 128, 16, False, True),                 # 40 rows of one token: a row tile's part
    ([3, 70], [200, 700], 40, 1, 64, 64, False, True),
    ([2], [130], 1024, 2, 64, 32, False, True),                       # more heads a group than rows a tile: of 256,
    ([1, 0, 0], [300, 0, 5], 40, 1, 128, 16, False, True),            # of 16
    ([200], [700], 4, 2, 128, 256, False, True),
    ([130, 140], [[130, 900], [257, 140]], 2, 2, 64, 256, True, False),
    ([300], [1], 2, 1, 128, 16, False, True),                         # a cache of one row: the last token sees it
    ([300], [1], 2, 1, 128, 16, False, False),
    ([500, 40], [20, 0], 2, 1, 64, 16, False, True),                  # chunks longer than their caches
    ([129, 257], [129, 257], 3, 3, 128, 128, False, True),
]
TAU = np.array([-1.5, 0.0, 2.0, 0.7, -0.25], dtype=np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_paged_attention_edges(dtype, case):
    n, lens, Hq, H, D, page, head, causal = CASES[case]
    rng = np.random.default_rng(500 + case)
    pg = Pages(rng, dtype, n, lens, H, D, page, head)
    q = rounded(rng.standard_normal((int(pg.cu[-1]) + 1, Hq, D)), dtype)
    tau = np.resize(TAU, Hq)
    out, lse = run_attention(pg, q, tau, causal)
    compare(pg, q, tau, causal, out, lse, dtype)


MANY = [
    # n, lens, Hq, H, D, page, head_pages: more sequences (and heads) than a block has threads
    ([i % 3 for i in range(900)], [1 + (i * 7) % 40 for i in range(900)], 2, 2, 64, 16, False),
    ([1] * 70, [[(b * 11 + h * 5) % 33 for h in range(9)] for b in range(70)], 9, 9, 64, 16, True),
    ([20] * 60, [[20 + (b + h) % 50 for h in range(12)] for b in range(60)], 24, 12, 64, 32, True),
    ([1], [3], 5000, 5000, 64, 16, False),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_sequences_and_heads(case):
    n, lens, Hq, H, D, page, head = MANY[case]
    rng = np.random.default_rng(700 + case)
    pg = Pages(rng, "bf16", n, lens, H, D, page, head)
    N = int(pg.cu[-1])
    q = rounded(rng.standard_normal((N, Hq, D)), "bf16")
    out, lse = run_attention(pg, q, None, True)
    compare(pg, q, None, True, out, lse, "bf16")
    d = pg.cuda()
    k, v = (rounded(rng.standard_normal((N, H, D)), "bf16").cuda() for _ in range(2))
    want = [d["k_pages"].clone(), d["v_pages"].clone()]
    for b in range(len(n)):
        for i in range(n[b]):
            for h in range(H if head else 1):
                at = ref.paged_row(pg.table, pg.lens, pg.cu, page, b, h, i)
                if at is None:
                    continue
                t = int(pg.cu[b]) + i
                for to, x in zip(want, (k, v)):
                    if head:
                        to[at] = x[t, h]
                    else:
                        to[at[0], :, at[1]] = x[t]
    st = status_word()
    vark.vark_paged_append(k, v, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                           vark.VARK_NORM_NONE, None, 0.0, None, None, st)
    check_status(st)
    assert same_bits(d["k_pages"], want[0]) and same_bits(d["v_pages"], want[1])


def test_broadcast_rows_are_read():
    """Strides of 0: one row for all heads, one token for all sequences."""
    rng = np.random.default_rng(3)
    pg = Pages(rng, "bf16", [2, 3], [40, 9], 4, 128, 16, False)
    one = rounded(rng.standard_normal((5, 1, 128)), "bf16").cuda()
    st = status_word()
    pools = []
    for k in (one.expand(5, 4, 128), one.expand(5, 4, 128).contiguous()):
        d = pg.cuda()
        vark.vark_paged_append(k, k, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                               vark.VARK_NORM_RMS, None, 1e-6, None, None, st)
        pools.append((d["k_pages"], d["v_pages"]))
    check_status(st)
    assert same_bits(pools[0][0], pools[1][0]) and same_bits(pools[0][1], pools[1][1])
    row = rounded(rng.standard_normal((1, 1, 128)), "bf16").cuda()
    d = pg.cuda()
    ws = torch.empty(vark.vark_paged_attention_workspace(5, 2, 8, 4, 128, 16, pg.table.shape[-1]), dtype=torch.uint8,
                     device="cuda")
    outs = []
    for q in (row.expand(5, 8, 128), row.expand(5, 8, 128).contiguous()):
        out = torch.empty(5, 8, 128, dtype=torch.bfloat16, device="cuda")
        vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"], None,
                                  True, out, None, ws, st)
        outs.append(out)
    check_status(st)
    assert same_bits(*outs)


def test_calls_with_nothing_to_do():
    rng = np.random.default_rng(1)
    bf, i32 = torch.bfloat16, torch.int32
    pg = Pages(rng, "bf16", [2, 1], [20, 3], 2, 64, 16, False)
    d = pg.cuda()
    st = status_word()
    ws = torch.empty(vark.vark_paged_attention_workspace(8, 2, 4, 2, 64, 16, 2), dtype=torch.uint8, device="cuda")
    rope = torch.from_numpy(rope_table(16, 64)).cuda()
    before = d["k_pages"].clone(), d["v_pages"].clone()

    def calls(n, cu, table, lens):
        q, k = (torch.ones(n, h, 64, dtype=bf, device="cuda") for h in (4, 2))
        out = torch.full_like(q, SENTINEL)
        lse = torch.full((n, 4), SENTINEL, device="cuda")
        pos = torch.full((n,), -1, dtype=i32, device="cuda")       # the chunk's tokens are padding
        x = [torch.full((1, n, h, 64), SENTINEL, dtype=bf, device="cuda") for h in (4, 2)]
        vark.vark_qk_norm_rope(q[None], k[None], *x, vark.VARK_NORM_RMS, None, None, 1e-6, rope, pos[None], st)
        vark.vark_paged_append(k, k, cu, d["k_pages"], d["v_pages"], table, lens, vark.VARK_NORM_RMS, None, 1e-6, rope,
                               pos, st)
        vark.vark_paged_attention(q, cu, d["k_pages"], d["v_pages"], table, lens, None, True, out, lse, ws, st)
        check_status(st)
        assert all((t == SENTINEL).all() for t in (out, lse, *x))
        assert same_bits(d["k_pages"], before[0]) and same_bits(d["v_pages"], before[1])

    zeros = torch.zeros(3, dtype=i32, device="cuda")
    calls(0, zeros, d["page_table"], d["cache_len"])               # no token
    calls(5, zeros, d["page_table"], d["cache_len"])               # padding only
    calls(5, zeros[:1], d["page_table"][:0], d["cache_len"][:0])   # no sequence
    calls(0, zeros[:1], d["page_table"][:0], d["cache_len"][:0])
    vark.vark_qk_norm_rope(None, torch.ones(0, 4, 2, 64, dtype=bf, device="cuda"), None,
                           torch.ones(0, 4, 2, 64, dtype=bf, device="cuda"), vark.VARK_NORM_L2, None, None, 1e-6, None,
                           None, st)
    check_status(st)


@pytest.mark.parametrize("head", [False, True])
def test_append_offsets_outside_the_chunk_are_recorded_and_skipped(head):
    rng = np.random.default_rng(2)
    n = [3, 0, 4, 2] + [1] * 40
    B, H = len(n), 2
    lens = np.repeat(np.array(n)[:, None] + 5, H, 1) if head else np.array(n) + 5
    pg = Pages(rng, "bf16", n, lens, H, 64, 16, head)
    N = int(pg.cu[-1])
    k = rounded(rng.standard_normal((N, H, 64)), "bf16").cuda()
    # (an entry of the tables, its new value, sequences whose tokens are not stored)
    for key, b, value, lost in (("cu_tokens", B, N + 9, [B - 1]), ("cu_tokens", 0, -2, [0]), ("cu_tokens", 2, 1, None),
                                ("cu_tokens", 41, N + 1, None), ("cache_len", 2, -1, [2]),
                                ("cache_len", 3, 10 ** 9, [3]), ("cache_len", 3, 2 ** 31 - 1, [3])):
        d = pg.cuda()
        d[key][b] = value
        before = d["k_pages"].clone()
        st = status_word()
        vark.vark_paged_append(k, k, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                               vark.VARK_NORM_NONE, None, 0.0, None, None, st)
        torch.cuda.synchronize()
        assert int(st.item()) == -2, (key, b)
        if lost is None:
            continue
        for s in range(B):
            for i in range(n[s]):
                for h in range(H):
                    at = ref.paged_row(pg.table, pg.lens, pg.cu, 16, s, h, i)
                    row = at if head else (at[0], h, at[1])
                    want = before[row] if s in lost else k[int(pg.cu[s]) + i, h]
                    assert same_bits(d["k_pages"][row], want), (key, b, s, i, h)
                    d["k_pages"][row] = before[row]
        assert same_bits(d["k_pages"], before)


def test_sequences_share_pages_that_are_read():
    """A prefix in the same pages for all, their own pages behind it."""
    rng = np.random.default_rng(6)
    for n in ([1, 2, 1], [150, 90, 200]):
        pg = Pages(rng, "bf16", n, [64 + 230] * 3, 2, 128, 32, False)
        pg.table[1, :2] = pg.table[2, :2] = pg.table[0, :2]
        q = rounded(rng.standard_normal((int(pg.cu[-1]), 4, 128)), "bf16")
        out, lse = run_attention(pg, q, None, True)
        compare(pg, q, None, True, out, lse, "bf16")


def test_lse_combines_disjoint_caches():
    """Attention over two halves of a cache, joined by their lse, is attention over the whole."""
    rng = np.random.default_rng(7)
    for n in ([1, 3], [100, 64]):
        whole = Pages(rng, "bf16", n, [512, 512], 2, 64, 64, False)
        q = rounded(rng.standard_normal((int(whole.cu[-1]), 4, 64)), "bf16")
        halves = []
        for i in range(2):
            part = Pages.__new__(Pages)
            part.__dict__.update(whole.__dict__, table=whole.table[:, 4 * i:4 * i + 4].copy(),
                                 lens=np.array([256, 256], dtype=np.int32))
            out, lse = run_attention(part, q, None, False)
            compare(part, q, None, False, out, lse, "bf16")
            halves.append((values(out), values(lse)))
        z = np.logaddexp(halves[0][1], halves[1][1])
        o = sum(v * np.exp(x - z)[..., None] for v, x in halves)
        want, lse, mean_abs, logit_abs = ref.paged_attention(values(q), whole.cu, values(whole.k), values(whole.v),
                                                             whole.table, whole.lens, np.ones(4, dtype=np.float32),
                                                             False)
        b_out, b_lse = attention_bounds(want, lse, mean_abs, logit_abs, 512.0, "bf16", 64)
        # each half's output is off by its own bound, its lse (and so its weight, relatively) by b_lse
        assert (np.abs(z - lse) <= b_lse).all()
        half_bounds = b_out + 2.0 ** -8 * sum(np.abs(v) * np.exp(x - z)[..., None] for v, x in halves)
        assert (np.abs(o - want) <= half_bounds + 2 * b_lse[..., None] * mean_abs).all()


@pytest.mark.parametrize("n", [[1, 1, 1], [70, 100, 60]])
def test_tables_written_on_the_stream_just_before(n):
    """Lengths, offsets and pages change on the stream between calls that
    follow one another without a host wait; a call sees those of its place."""
    rng = np.random.default_rng(9)
    pg = Pages(rng, "bf16", n, [900, 1300, 400], 2, 64, 16, False)
    N = int(pg.cu[-1])
    q = rounded(rng.standard_normal((N, 8, 64)), "bf16").cuda()
    d = pg.cuda()
    ws = torch.empty(vark.vark_paged_attention_workspace(N, 3, 8, 2, 64, 16, pg.table.shape[-1]), dtype=torch.uint8,
                     device="cuda")
    st = status_word()
    steps = 60
    lens = torch.from_numpy(np.maximum(pg.lens[None] - rng.integers(0, 300, (steps, 3)), 1).astype(np.int32)).cuda()
    out = torch.empty(steps, N, 8, 64, dtype=torch.bfloat16, device="cuda")
    want = torch.empty_like(out)

    def step(i, to):
        d["cache_len"].copy_(lens[i])
        vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"], None,
                                  True, to, None, ws, st)

    for i in range(steps):
        step(i, want[i])
        torch.cuda.synchronize()
    for i in range(steps):
        step(i, out[i])
    check_status(st)
    assert same_bits(out, want)


@pytest.mark.parametrize("head", [False, True])
def test_both_ways_through_the_binding(head, monkeypatch):
    """The marshalling module and the Python functions behind it make the same calls."""
    assert vark._quick(), "the module _paged_call is not built"
    rng = np.random.default_rng(12)
    n, H, D, ps = [3, 1, 20], 2, 128, 32
    pg = Pages(rng, "bf16", n, [[40, 3], [1, 9], [300, 20]] if head else [40, 1, 300], H, D, ps, head)
    N = int(pg.cu[-1])
    qkv = rounded(rng.standard_normal((1, N, 4 + 2 * H, D)), "bf16").cuda()
    rope = torch.from_numpy(rope_table(400, 64)).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    weight = torch.rand(D, device="cuda")
    tau = torch.from_numpy(rng.uniform(0.5, 2, 4).astype(np.float32)).cuda()
    ws = torch.empty(vark.vark_paged_attention_workspace(N, 3, 4, H, D, ps, pg.table.shape[-1]), dtype=torch.uint8,
                     device="cuda")
    st = status_word()
    got = []
    for quick in (vark._quick(), False):
        monkeypatch.setattr(vark, "_quick_module", quick)
        d = pg.cuda()
        q = torch.empty(4, N, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        k = torch.empty(1, N, H, D, dtype=torch.bfloat16, device="cuda")
        vark.vark_qk_norm_rope(qkv[:, :, :4], qkv[:, :, 4:4 + H], q[None], k, vark.VARK_NORM_L2, weight, None, 1e-6,
                               rope, pos[None], st, pairs=True)
        vark.vark_paged_append(qkv[0, :, 4:4 + H], qkv[0, :, 4 + H:], d["cu_tokens"], d["k_pages"], d["v_pages"],
                               d["page_table"], d["cache_len"], vark.VARK_NORM_RMS, weight, 1e-6, rope, pos, st,
                               stream=torch.cuda.current_stream().cuda_stream)
        out = torch.empty(N, 4, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(N, 4, device="cuda")
        vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"], tau,
                                  head, out, lse, ws, st, stream=torch.cuda.current_stream())
        check_status(st)
        got.append((q, k, d["k_pages"], d["v_pages"], out, lse.view(torch.bfloat16)))
        for call in (lambda: vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                                                       d["cache_len"], tau, head, q, lse, ws, st),
                     lambda: vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                                                       d["cache_len"], tau, head, out[:1].expand(N, 4, D), lse, ws, st),
                     lambda: vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                                                       d["cache_len"], tau[:3], head, out, lse, ws, st)):
            with pytest.raises(ValueError):
                call()
        with pytest.raises(vark.VarkError):
            vark.vark_paged_attention(q, d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                                      tau, head, out, lse, ws[:16], st)
    for a, b in zip(*got):
        assert same_bits(a, b)
