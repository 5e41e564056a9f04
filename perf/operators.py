"""What is measured of the serving operators: norm + rotation of queries and
keys, the append to a paged cache, and attention of a chunk over that cache.

`run` computes them in elementary torch operations (own = False) or through
the library's calls (own = True); `exact` gives the values in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_NORMS = {"none": 0, "rms": 1, "l2": 2}
_EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _norm_rope(name, **kw):
    c = dict(op="norm_rope", name=name, dtype="bf16", B=1, T=1, Hq=32, Hkv=8, D=128, norm="rms", weight=True,
             rope_dim=128, pairs=False, layout="token", rope_len=16384)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(op="append", name=name, dtype="bf16", B=1, Hkv=8, D=128, page=64, head_pages=False, q_lo=1, q_hi=1,
             past_lo=0, past_hi=1000, len_seed=1, norm="rms", rope_dim=128, pairs=False, pad=0, rope_len=16384)
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(op="attention", name=name, dtype="bf16", B=1, Hq=32, Hkv=8, D=128, page=64, head_pages=False, q_lo=1,
             q_hi=1, past_lo=0, past_hi=1000, len_seed=1, causal=True, pad=0)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of a small batch: latency
        _norm_rope("norm_rope_decode_b8", T=8),
        # the queries and keys of the last scale (64 x 64 tokens) of a batch of 8, unit length and 2-D rotation, written
        # head-major for the dense attention calls
        _norm_rope("norm_rope_scale12_head_major", B=8, T=4096, Hq=16, Hkv=16, norm="l2", weight=False,
                   layout="head", rope_len=10521),
        # a long chunk read out of a fused projection's output, half of the channels rotated in adjacent pairs
        _norm_rope("norm_rope_fused_fp16", dtype="fp16", T=8191, D=64, Hq=32, Hkv=8, rope_dim=32, pairs=True,
                   layout="fused"),
        # one decoding step of 64 sequences
        _append("append_decode_b64", B=64, past_lo=1, past_hi=1023, page=16),
        # ragged chunks of 8 sequences, some padding behind the last
        _append("append_chunks_ragged", B=8, q_lo=301, q_hi=2047, past_lo=0, past_hi=999, pad=13),
        # the last scale's keys and values behind each head's own retained past
        _append("append_scale12_head_pages", B=4, Hkv=16, q_lo=4096, q_hi=4096, past_lo=5, past_hi=2500,
                head_pages=True, norm="l2", page=128, rope_len=10521),
        # decoding one sequence with a long cache
        _attn("attn_decode_b1_64k", past_lo=65536, past_hi=65536),
        # decoding a ragged batch out of small pages
        _attn("attn_decode_b64_ragged", B=64, past_lo=3, past_hi=8190, page=16),
        # drafted tokens checked in one pass
        _attn("attn_drafts_fp16", dtype="fp16", B=32, q_lo=3, q_hi=7, past_lo=100, past_hi=4000, D=64, Hq=24, Hkv=8,
              page=32),
        # one long prompt taken in chunks: a chunk over the cache so far
        _attn("attn_chunk_2048_over_16k", q_lo=2048, q_hi=2048, past_lo=16384, past_hi=16384, page=128),
        # first chunks of a ragged batch
        _attn("attn_prompts_ragged", B=8, q_lo=333, q_hi=4099, past_lo=0, past_hi=0, page=16, pad=5),
        # the last scale of a batch of 8 over each head's own retained past: every new token sees the whole scale
        _attn("attn_scale12_head_pages", B=8, Hq=16, Hkv=16, q_lo=4096, q_hi=4096, past_lo=5, past_hi=2500,
              causal=False, head_pages=True, page=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    largest = {}
    for c in listed():
        w = work(c)
        for k in w:
            largest[k] = max(largest.get(k, 0), w[k])
    while True:
        op = rng.choice(["norm_rope", "append", "attention", "attention"])
        D = rng.choice([64, 128])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        page = rng.choice([16, 32, 64, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8, 16])
        G = rng.choice([1, 2, 3, 4, 5, 8, 16])
        seed = rng.randrange(1 << 30)
        norm = rng.choice(["none", "rms", "l2"])
        rope = rng.choice([16 * i for i in range(D // 16 + 1)])
        pairs = rng.random() < 0.5
        B = _log_int(rng, 1, 96)
        pad = rng.choice([0, 0, 1, 17])
        kind = rng.choice(["one", "few", "chunk"])
        q_hi = {"one": 1, "few": rng.randint(2, 8), "chunk": _log_int(rng, 9, 5000)}[kind]
        q_lo = max(1, q_hi - rng.randrange(q_hi))
        past_hi = _log_int(rng, 1, 66000) if B < 8 else _log_int(rng, 1, 8000)
        past_lo = rng.randint(0, past_hi)
        head_pages = rng.random() < 0.3
        if op == "norm_rope":
            c = _norm_rope("", dtype=dtype, B=rng.randint(1, 8), T=_log_int(rng, 1, 10000), Hq=Hkv * G, Hkv=Hkv, D=D,
                           norm=norm, weight=rng.random() < 0.7, rope_dim=rope, pairs=pairs,
                           layout=rng.choice(["token", "head", "fused"]))
        elif op == "append":
            past_hi = min(past_hi, 2500)
            past_lo = min(past_lo, past_hi)
            c = _append("", dtype=dtype, B=B, Hkv=Hkv, D=D, page=page, head_pages=head_pages, q_lo=q_lo, q_hi=q_hi,
                        past_lo=past_lo, past_hi=past_hi, len_seed=seed, norm=norm, rope_dim=rope, pairs=pairs, pad=pad)
            if B * Hkv * D * (past_hi + q_hi + page) > (1 << 27):
                continue
        else:
            c = _attn("", dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, head_pages=head_pages, q_lo=q_lo,
                      q_hi=q_hi, past_lo=past_lo, past_hi=past_hi, len_seed=seed, causal=rng.random() < 0.7, pad=pad)
        del c["name"]
        w = work(c)
        if all(w[k] <= largest[k] for k in w):
            return c


def _lengths(case):
    """Tokens of every sequence, and past rows of every (sequence, table head)."""
    rng = random.Random(case["len_seed"])
    n_tab = case["Hkv"] if case["head_pages"] else 1
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    past = [[rng.randint(case["past_lo"], case["past_hi"]) for _ in range(n_tab)] for _ in range(case["B"])]
    return q, past


def _seen(case, q, past):
    """Keys seen by the q queries of a sequence, summed over the queries."""
    return q * past + (q * (q + 1) // 2 if case["causal"] else q * q)


def work(case):
    D = case["D"]
    if case["op"] == "norm_rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hkv"]) * D
        per = (4 if case["norm"] != "none" else 0) + (3 if case["rope_dim"] else 0)
        return {"bytes": 4 * n, "flops": per * n}
    q, past = _lengths(case)
    if case["op"] == "append":
        n = sum(q) * case["Hkv"] * D
        per = (4 if case["norm"] != "none" else 0) + (3 if case["rope_dim"] else 0)
        return {"bytes": 8 * n, "flops": per * n}
    rep = 1 if case["head_pages"] else case["Hkv"]
    G = case["Hq"] // case["Hkv"]
    rows = sum(q) * case["Hq"]
    kv = sum((p + n) * rep for n, ps in zip(q, past) for p in ps)
    seen = sum(_seen(case, n, p) * rep for n, ps in zip(q, past) for p in ps)
    return {"bytes": rows * (4 * D + 4) + 4 * D * kv, "flops": 4 * D * G * seen}


# ------------------------------------------------------------------ inputs
def _rope_table(case):
    """[rope_len][2][R / 2] cosines and sines; None without a rotation."""
    R, n = case["rope_dim"], case["rope_len"]
    if R == 0:
        return None
    pos = torch.arange(n, device="cuda", dtype=torch.float64)
    freq = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float64) * 2.0 / R)
    ang = pos[:, None] * freq[None, :]
    return torch.stack([ang.cos(), ang.sin()], dim=1).float().contiguous()


def _prepare_norm_rope(case, g):
    dt = _DTYPES[case["dtype"]]
    B, T, Hq, Hk, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").mul_(1.5).to(dt)

    if case["layout"] == "fused":
        qkv = rnd(B, T, Hq + 2 * Hk, D)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    else:
        q, k = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
    if case["layout"] == "head":
        q_out = torch.zeros(B, Hq, T, D, dtype=dt, device="cuda").transpose(1, 2)
        k_out = torch.zeros(B, Hk, T, D, dtype=dt, device="cuda").transpose(1, 2)
    else:
        q_out = torch.zeros(B, T, Hq, D, dtype=dt, device="cuda")
        k_out = torch.zeros(B, T, Hk, D, dtype=dt, device="cuda")
    s = dict(q=q, k=k, q_out=q_out, k_out=k_out, qw=None, kw=None)
    if case["weight"] and case["norm"] != "none":
        s["qw"] = torch.rand(D, generator=g, device="cuda") + 0.5
        s["kw"] = torch.rand(D, generator=g, device="cuda") + 0.5
    first = torch.randint(0, max(1, case["rope_len"] - T), (B, 1), generator=g, device="cuda")
    pos = (first + torch.arange(T, device="cuda")[None]) % case["rope_len"]
    s["positions"] = pos.to(torch.int32).contiguous() if case["rope_dim"] else None
    return s


def _prepare_pages(case, g):
    """Cache, tables and lengths; every sequence's pages lie scattered."""
    dt = _DTYPES[case["dtype"]]
    B, H, D, ps = case["B"], case["Hkv"], case["D"], case["page"]
    q, past = _lengths(case)
    need = [[-(-(p + n) // ps) for p in pb] for n, pb in zip(q, past)]
    width = max(max(r) for r in need)
    total = sum(sum(r) for r in need)
    n_pages = total + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((B, len(past[0]), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        for t in range(len(past[0])):
            table[b, t, :need[b][t]] = perm[at:at + need[b][t]]
            at += need[b][t]
    shape = (n_pages, ps, D) if case["head_pages"] else (n_pages, H, ps, D)

    def rnd(*shape):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)

    lens = torch.tensor([[p + n for p in pb] for n, pb in zip(q, past)], dtype=torch.int32, device="cuda")
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    s = dict(k_pages=rnd(*shape), v_pages=rnd(*shape), q_len=q, past=past, cu=cu, N=cu[-1] + case["pad"],
             cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             page_table=table if case["head_pages"] else table[:, 0].contiguous(),
             cache_len=lens if case["head_pages"] else lens[:, 0].contiguous(), rnd=rnd)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "norm_rope":
        s = _prepare_norm_rope(case, g)
    else:
        s = _prepare_pages(case, g)
        rnd, N, H, D = s.pop("rnd"), s["N"], case["Hkv"], case["D"]
        if case["op"] == "append":
            s["k"], s["v"] = rnd(N, H, D).mul_(1.5), rnd(N, H, D)
            s["kw"] = torch.rand(D, generator=g, device="cuda") + 0.5 if case["norm"] != "none" else None
            pos = torch.zeros(N, dtype=torch.int32)
            for b, n in enumerate(s["q_len"]):
                pos[s["cu"][b]:s["cu"][b] + n] = torch.arange(n) + s["past"][b][0]
            s["positions"] = (pos % case["rope_len"]).to("cuda", torch.int32) if case["rope_dim"] else None
        else:
            s["q"] = rnd(N, case["Hq"], D)
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(N, case["Hq"], device="cuda")
            s["tau"] = torch.rand(case["Hq"], generator=g, device="cuda") * 1.5 + 0.5
    s["rope"] = _rope_table(case) if case["op"] != "attention" else None
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["case"] = dict(case)
    if own:
        import kv_cache_compression_cas_b200 as vark
        s["vark"] = vark
        if case["op"] == "attention":
            n = vark.vark_paged_attention_workspace(s["N"], case["B"], case["Hq"], case["Hkv"], case["D"], case["page"],
                                                    s["page_table"].shape[-1])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms
def _norm_rotate(x, norm, w, table, positions, pairs):
    """x [..., H, D] in 32 bits; positions [...] or None."""
    D = x.shape[-1]
    if norm == "rms":
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + _EPS)
    elif norm == "l2":
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True)).clamp_min(_EPS)
    if w is not None:
        x = x * w
    if table is None:
        return x
    cs = table[positions.long()].unsqueeze(-3)
    c, s = cs[..., 0, :], cs[..., 1, :]
    R = 2 * c.shape[-1]
    if pairs:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        rot = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        rot = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([rot, x[..., R:]], dim=-1)


def _plain_norm_rope(s):
    c = s["case"]
    for x, w, o in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
        o.copy_(_norm_rotate(x.float(), c["norm"], w, s["rope"], s["positions"], c["pairs"]))
    return s["q_out"], s["k_out"]


def _plain_append(s):
    c = s["case"]
    n = s["cu"][-1]
    ps = c["page"]
    k = _norm_rotate(s["k"][:n].float(), c["norm"], s["kw"], s["rope"],
                     None if s["positions"] is None else s["positions"][:n], c["pairs"]).to(s["k"].dtype)
    v = s["v"][:n]
    dev = k.device
    cu = s["cu_tokens"].long()
    tok = torch.arange(n, device=dev)
    b = torch.searchsorted(cu, tok, right=True) - 1
    b = b.clamp_max(c["B"] - 1)
    q_len = cu[1:] - cu[:-1]
    if c["head_pages"]:
        row = s["cache_len"][b].long() - q_len[b][:, None] + (tok - cu[b])[:, None]          # [n][H]
        page = s["page_table"][b].long().gather(2, (row // ps)[..., None])[..., 0]
        s["k_pages"][page, row % ps] = k
        s["v_pages"][page, row % ps] = v
    else:
        row = s["cache_len"][b].long() - q_len[b] + tok - cu[b]                              # [n]
        page = s["page_table"][b, row // ps].long()
        s["k_pages"][page, :, row % ps] = k
        s["v_pages"][page, :, row % ps] = v
    return s["k_pages"], s["v_pages"]


def _rows(pages, table, head):
    """Rows of table [B][P], or of head-specific table [B][H][P]: [B][H][P * page][D] in 32 bits."""
    ids = table.long().clamp_min(0)
    if head:
        return pages[ids].flatten(2, 3).float()
    return pages[ids].transpose(1, 2).flatten(2, 3).float()


def _attend(q, K, V, keys, lim):
    """q [B][H][R][D], K and V [B][H][L][D], keys [B][H] rows that count of them (others may hold anything), lim
    [B][H][R] of those that row r sees: outputs [B][H][R][D] and log-sums [B][H][R]."""
    j = torch.arange(K.shape[2], device=K.device)
    V = V.masked_fill((j >= keys[..., None])[..., None], 0.0)
    x = q @ K.transpose(-1, -2)
    x.masked_fill_(j >= lim[..., None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    return (x @ V) / l, (m + l.log())[..., 0]


def _plain_attention(s):
    """A batch of few tokens each in one padded pass, chunks of many sequence by sequence."""
    c = s["case"]
    D, H, ps, B = c["D"], c["Hkv"], c["page"], c["B"]
    G = c["Hq"] // H
    qs = s["q"].float() * (s["tau"] / math.sqrt(D))[:, None]
    cu = s["cu_tokens"].long()
    n_tok = cu[1:] - cu[:-1]
    lens = s["cache_len"].long().view(B, -1).expand(B, H)                                   # [B][H]
    most = max(s["q_len"])
    spans = [(0, B)] if most * G <= 64 else [(b, b + 1) for b in range(B)]
    for b0, b1 in spans:
        n = max(s["q_len"][b0:b1])
        pages = -(-max(max(s["past"][b]) + s["q_len"][b] for b in range(b0, b1)) // ps)
        K = _rows(s["k_pages"], s["page_table"][b0:b1, ..., :pages], c["head_pages"])
        V = _rows(s["v_pages"], s["page_table"][b0:b1, ..., :pages], c["head_pages"])
        i = torch.arange(n, device=K.device)
        real = i < n_tok[b0:b1, None]                                                       # [b][n]
        tok = (cu[b0:b1, None] + i).clamp_max(cu[-1] - 1)
        q = qs[tok].view(b1 - b0, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(b1 - b0, H, G * n, D)
        length = lens[b0:b1]
        if c["causal"]:
            lim = torch.minimum(length[..., None] - n_tok[b0:b1, None, None] + i + 1, length[..., None])
        else:
            lim = length[..., None].expand(-1, -1, n)
        lim = lim.repeat(1, 1, G)                                                           # rows: g * n + i
        step = max(1, min(H, (1 << 30) // (q.shape[0] * q.shape[2] * K.shape[2])))
        done = [_attend(q[:, h:h + step], K[:, h:h + step], V[:, h:h + step], length[:, h:h + step],
                        lim[:, h:h + step]) for h in range(0, H, step)]
        o = torch.cat([d[0] for d in done], 1).view(-1, H, G, n, D).permute(0, 3, 1, 2, 4).flatten(2, 3)
        z = torch.cat([d[1] for d in done], 1).view(-1, H, G, n).permute(0, 3, 1, 2).flatten(2, 3)
        s["out"][tok[real]] = o[real].to(s["out"].dtype)
        s["lse"][tok[real]] = z[real]
    return s["out"], s["lse"]


# ------------------------------------------------------------------ the library's calls
def _own(s):
    c, vark = s["case"], s["vark"]
    if c["op"] == "norm_rope":
        vark.vark_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], _NORMS[c["norm"]], s["qw"], s["kw"], _EPS,
                               s["rope"], s["positions"], s["status"], pairs=c["pairs"])
        return s["q_out"], s["k_out"]
    if c["op"] == "append":
        vark.vark_paged_append(s["k"], s["v"], s["cu_tokens"], s["k_pages"], s["v_pages"], s["page_table"],
                               s["cache_len"], _NORMS[c["norm"]], s["kw"], _EPS, s["rope"], s["positions"],
                               s["status"], pairs=c["pairs"])
        return s["k_pages"], s["v_pages"]
    vark.vark_paged_attention(s["q"], s["cu_tokens"], s["k_pages"], s["v_pages"], s["page_table"], s["cache_len"],
                              s["tau"], c["causal"], s["out"], s["lse"], s["workspace"], s["status"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append,
            "attention": _plain_attention}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(x, c, w, table, positions):
    """Norm and rotation of x [n][H][D], one channel pair after another."""
    y = x.double()
    if c["norm"] == "rms":
        y = y * torch.rsqrt(y.square().mean(dim=2, keepdim=True) + _EPS)
    elif c["norm"] == "l2":
        y = y / torch.linalg.vector_norm(y, dim=2, keepdim=True).clamp(min=_EPS)
    if w is not None:
        y = torch.einsum("nhd,d->nhd", y, w.double())
    if table is not None:
        half = table.shape[2]
        t = table.double().index_select(0, positions.long())
        z = y.clone()
        for j in range(half):
            i0, i1 = (2 * j, 2 * j + 1) if c["pairs"] else (j, j + half)
            co, si = t[:, 0, j, None], t[:, 1, j, None]
            z[:, :, i0] = y[:, :, i0] * co - y[:, :, i1] * si
            z[:, :, i1] = y[:, :, i1] * co + y[:, :, i0] * si
        y = z
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm_rope":
        outs = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            rows = x.flatten(0, 1)
            p = None if s["positions"] is None else s["positions"].flatten()
            outs.append(_exact_rows(rows, c, w, s["rope"], p).view(x.shape))
        return tuple(outs)
    H, D, ps = c["Hkv"], c["D"], c["page"]
    if c["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        k = _exact_rows(s["k"], c, s["kw"], s["rope"], s["positions"])
        for b, n in enumerate(s["q_len"]):
            new_k, new_v = k[s["cu"][b]:s["cu"][b + 1]], s["v"][s["cu"][b]:s["cu"][b + 1]].double()
            for t, past in enumerate(s["past"][b]):
                ids = (s["page_table"][b, t] if c["head_pages"] else s["page_table"][b]).tolist()
                r = past
                while r < past + n:                      # page by page
                    e = min(past + n, (r // ps + 1) * ps)
                    for pool, new in ((kp, new_k), (vp, new_v)):
                        if c["head_pages"]:
                            pool[ids[r // ps], r % ps:r % ps + e - r] = new[r - past:e - past, t]
                        else:
                            pool[ids[r // ps], :, r % ps:r % ps + e - r] = new[r - past:e - past].transpose(0, 1)
                    r = e
        return kp, vp
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    G = c["Hq"] // H
    for b, n in enumerate(s["q_len"]):
        for h in range(H):
            length = s["past"][b][h if c["head_pages"] else 0] + n
            ids = (s["page_table"][b, h] if c["head_pages"] else s["page_table"][b])[:-(-length // ps)].long()
            pool = (lambda t: t[ids] if c["head_pages"] else t[ids, h])
            K = pool(s["k_pages"]).reshape(-1, D)[:length].double()
            V = pool(s["v_pages"]).reshape(-1, D)[:length].double()
            for hq in range(h * G, (h + 1) * G):
                for r0 in range(0, n, 2048):
                    r1 = min(n, r0 + 2048)
                    rows = slice(s["cu"][b] + r0, s["cu"][b] + r1)
                    x = torch.einsum("rd,kd->rk", s["q"][rows, hq].double(), K) * (float(s["tau"][hq]) * D ** -0.5)
                    if c["causal"]:
                        x = x.tril(length - n + r0).masked_fill(
                            torch.ones_like(x, dtype=torch.bool).triu(length - n + r0 + 1), -math.inf)
                    z = torch.logsumexp(x, dim=1)
                    lse[rows, hq] = z
                    out[rows, hq] = torch.exp(x - z[:, None]) @ V
    return out, lse
