"""Refusals of the serving calls, before any device work: status codes of the C
ABI and exceptions of the binding; and pins of the oracle they are tested
against."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from oracle import paged as ref

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


S3, S2 = strides(4096, 512, 128), strides(512, 128)
NO_DEVICE = (-7, -5)       # the checks passed: there is no device here


def norm_rope(**kw):
    a = dict(dtype=0, q=P, qs=S3, qo=P, qos=S3, Hq=4, k=P, ks=S3, ko=P, kos=S3, Hk=2, B=1, T=3, D=128, norm=1, qw=P,
             kw=P, eps=1e-6, rope=P, rope_len=10, rope_dim=64, pairs=0, pos=P, st=P, stream=None)
    a.update(kw)
    return vark.library().vark_qk_norm_rope(*a.values())


def append(**kw):
    a = dict(dtype=0, k=P, ks=S2, v=P, vs=S2, n=5, B=2, H=4, D=128, cu=P, kp=P, vp=P, n_pages=7, page=16, table=P,
             max_pages=3, lens=P, head=0, norm=1, w=P, eps=1e-6, rope=P, rope_len=10, rope_dim=64, pairs=0, pos=P,
             st=P, stream=None)
    a.update(kw)
    return vark.library().vark_paged_append(*a.values())


def attention(**kw):
    a = dict(dtype=0, q=P, qs=S2, n=5, B=2, Hq=8, H=4, D=128, cu=P, kp=P, vp=P, n_pages=7, page=16, table=P,
             max_pages=3, lens=P, head=0, tau=P, causal=1, out=P, os=S2, lse=P, ws=P, ws_bytes=1 << 40, st=P,
             stream=None)
    a.update(kw)
    return vark.library().vark_paged_attention(*a.values())


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: only where nothing can launch")
def test_status_codes():
    for call in (norm_rope, append, attention):
        assert call() in NO_DEVICE
        assert call(dtype=2) == -1
        assert call(st=None) == -1
        assert call(D=96) == -2
    # norm and rotation
    assert norm_rope(q=None, k=None) == -1
    assert norm_rope(q=None, qs=None, qo=None, qos=None, Hq=0, qw=None) in NO_DEVICE
    assert norm_rope(qo=None) == -1 and norm_rope(kos=None) == -1
    assert norm_rope(norm=3) == -1 and norm_rope(eps=-1.0) == -1 and norm_rope(eps=math.nan) == -1
    assert norm_rope(rope=None) == -1 and norm_rope(pos=None) == -1
    assert norm_rope(rope=None, pos=None) in NO_DEVICE
    assert norm_rope(rope_dim=72) == -2 and norm_rope(rope_dim=144) == -2 and norm_rope(rope_len=0) == -2
    assert norm_rope(B=-1) == -2 and norm_rope(Hq=0) == -2 and norm_rope(T=-1) == -2
    assert norm_rope(qs=strides(4096, 516, 128)) == -3 and norm_rope(kos=strides(4096, -512, 128)) == -3
    assert norm_rope(qs=strides(-3, 512, 128)) in NO_DEVICE      # an axis of one entry has no step
    assert norm_rope(q=ODD) == -3 and norm_rope(qw=ODD) == -3 and norm_rope(rope=ODD) == -3
    # append
    for name in ("k", "ks", "v", "vs", "cu", "kp", "vp", "table", "lens"):
        assert append(**{name: None}) == -1
    assert append(page=24) == -2 and append(page=512) == -2 and append(n_pages=0) == -2 and append(max_pages=0) == -2
    assert append(max_pages=1 << 28) == -2            # rows of a cache are counted in 31 bits
    assert append(n=-1) == -2 and append(n=1 << 31) == -2 and append(H=0) == -2 and append(B=-1) == -2
    assert append(ks=strides(4, 128)) == -3 and append(vp=ODD) == -3
    # attention
    for name in ("q", "qs", "cu", "kp", "vp", "table", "lens", "out", "os", "ws"):
        assert attention(**{name: None}) == -1
    assert attention(tau=None, lse=None) in NO_DEVICE
    assert attention(Hq=6) == -2 and attention(Hq=2) == -2 and attention(H=0) == -2
    assert attention(n=1 << 30) == -2 and attention(B=1 << 24) == -2
    assert attention(page=8) == -2
    need = vark.vark_paged_attention_workspace(5, 2, 8, 4, 128, 16, 3)
    assert need > 0 and attention(ws_bytes=need) in NO_DEVICE and attention(ws_bytes=need - 1) == -1
    assert attention(ws=ODD) == -3 and attention(os=strides(512, 100)) == -3
    with pytest.raises(vark.VarkError):
        vark.vark_paged_attention_workspace(5, 2, 8, 3, 128, 16, 3)


def test_binding_refuses_mismatched_tensors():
    bf, i32 = torch.bfloat16, torch.int32
    B, T, Hq, Hk, D = 2, 3, 4, 2, 64
    q, k = torch.zeros(B, T, Hq, D, dtype=bf), torch.zeros(B, T, Hk, D, dtype=bf)
    st = torch.zeros(1, dtype=i32)
    good = dict(q=q, k=k, q_out=q, k_out=k, norm=1, q_weight=torch.ones(D), k_weight=None, eps=1e-6,
                rope=torch.zeros(9, 2, 16), positions=torch.zeros(B, T, dtype=i32), dev_status=st)
    for key, bad in (("k", k[:1]), ("q_out", q[:, :2]), ("q_weight", torch.ones(D + 1)), ("q_out", None),
                     ("rope", None), ("rope", torch.zeros(9, 3, 16)), ("positions", torch.zeros(5, dtype=i32)),
                     ("dev_status", torch.zeros(0, dtype=i32))):
        with pytest.raises(ValueError):
            vark.vark_qk_norm_rope(**{**good, key: bad})
    for key, bad in (("q", q.float()), ("k", k.half()), ("q", q), ("rope", torch.zeros(9, 2, 16).double())):
        with pytest.raises(TypeError):         # the last good one: CPU tensors
            vark.vark_qk_norm_rope(**{**good, key: bad})
    n, H, ps, P_ = 5, 2, 16, 7
    pool = torch.zeros(P_, H, ps, D, dtype=bf)
    kv = torch.zeros(n, H, D, dtype=bf)
    base = dict(cu_tokens=torch.zeros(3, dtype=i32), k_pages=pool, v_pages=pool,
                page_table=torch.zeros(2, 4, dtype=i32), cache_len=torch.zeros(2, dtype=i32), dev_status=st)
    app = dict(base, k=kv, v=kv, norm=0, k_weight=None, eps=0.0, rope=None, positions=None)
    att = dict(base, q=torch.zeros(n, 4, D, dtype=bf), tau=torch.ones(4), causal=True,
               out=torch.zeros(n, 4, D, dtype=bf), lse=torch.zeros(n, 4), workspace=torch.zeros(8, dtype=torch.uint8))
    for call, args in ((vark.vark_paged_append, app), (vark.vark_paged_attention, att)):
        for key, bad in (("v_pages", pool[:-1]), ("page_table", torch.zeros(3, 4, dtype=i32)),
                         ("page_table", torch.zeros(2, 2, 4, dtype=i32)), ("cache_len", torch.zeros(2, 2, dtype=i32)),
                         ("cu_tokens", torch.zeros(0, dtype=i32)), ("k_pages", pool[:, 0])):
            with pytest.raises(ValueError):
                call(**{**args, key: bad})
        with pytest.raises(TypeError):
            call(**args)
    for key, bad in (("v", kv[:4]), ("k_weight", torch.ones(3)), ("positions", torch.zeros(n, dtype=i32))):
        with pytest.raises(ValueError):
            vark.vark_paged_append(**{**app, key: bad})
    for key, bad in (("out", torch.zeros(n, 3, D, dtype=bf)), ("lse", torch.zeros(n, 3)), ("tau", torch.ones(3)),
                     ("q", torch.zeros(n, 3, D, dtype=bf))):
        with pytest.raises(ValueError):
            vark.vark_paged_attention(**{**att, key: bad})


# ------------------------------------------------------------------ oracle pins
def test_oracle_norm_rotate_closed_forms():
    x = np.zeros((2, 1, 16))
    x[0, 0, 0], x[0, 0, 8] = 3.0, 4.0
    x[1, 0, :2] = (5.0, 12.0)
    quarter = np.stack([np.zeros((2, 8)), np.ones((2, 8))], axis=1).astype(np.float32)     # cos 0, sin 1
    y, _ = ref.norm_rotate(x[:1], ref.NORM_L2, None, 1e-6, quarter, [1], False)
    assert np.allclose(y[0, 0, [0, 8]], [-0.8, 0.6])          # (a, b) -> (-b, a), unit length
    y, _ = ref.norm_rotate(x[1:], ref.NORM_RMS, np.arange(16.0), 0.0, quarter, [0], True)
    rms = 13.0 / 4.0
    assert np.allclose(y[0, 0, :2], [-12.0 / rms, 0.0])       # weight 0 on the first channel
    y, _ = ref.norm_rotate(x, ref.NORM_NONE, None, 0.0, None, None, False)
    assert np.array_equal(y, x)


@pytest.mark.parametrize("causal", [True, False])
def test_oracle_paged_attention_is_softmax_attention(causal):
    """Against torch's fp64 attention with an explicit mask, and uniform
    weights against plain means."""
    rng = np.random.default_rng(2)
    H, G, D, ps = 2, 3, 16, 4
    n, length = 5, 11
    pool_k, pool_v = rng.standard_normal((2, 9, H, ps, D))
    table, lens, cu = np.array([[7, 2, 5]]), np.array([length]), np.array([0, n])
    q = rng.standard_normal((n, H * G, D))
    tau = rng.uniform(0.5, 2, H * G)
    out, lse, _, _ = ref.paged_attention(q, cu, pool_k, pool_v, table, lens, tau, causal)
    rows = [(table[0, r // ps], r % ps) for r in range(length)]
    K = np.stack([[pool_k[p, h, r] for p, r in rows] for h in range(H)]).repeat(G, axis=0)
    V = np.stack([[pool_v[p, h, r] for p, r in rows] for h in range(H)]).repeat(G, axis=0)
    mask = torch.ones(n, length, dtype=torch.bool)
    if causal:
        mask = mask.tril(length - n)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q.transpose(1, 0, 2) * tau[:, None, None]), torch.from_numpy(K), torch.from_numpy(V),
        attn_mask=mask)
    assert np.allclose(out.transpose(1, 0, 2), want.numpy(), atol=1e-12)
    out, lse, _, _ = ref.paged_attention(np.zeros_like(q), cu, pool_k, pool_v, table, lens, tau, causal)
    seen = [length - n + i + 1 if causal else length for i in range(n)]
    for i in range(n):
        assert np.allclose(lse[i], math.log(seen[i]))
        assert np.allclose(out[i, 0], V[0, :seen[i]].mean(0))


def test_oracle_rows_of_a_cache_shorter_than_its_chunk():
    table, cu = np.array([[3, 1]]), np.array([0, 6])
    assert ref.paged_row(table, np.array([4]), cu, 2, 0, 0, 1) is None
    assert ref.paged_row(table, np.array([4]), cu, 2, 0, 0, 2) == (3, 0)
    assert ref.paged_row(table, np.array([4]), cu, 2, 0, 0, 5) == (1, 1)
