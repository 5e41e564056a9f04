"""Random paged-cache problems for the tests: inputs as bits, tables, and the
rounding bounds that the comparisons use.  No step of the method is computed
here."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# half a step of the type, relative to the value; of fp32
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
U32 = 2.0 ** -24
# below this an fp16 value's step no longer shrinks: half of 2^-24
FP16_TINY = 2.0 ** -25


def rounded(x, dtype):
    """A CPU tensor of the type, from fp64 values."""
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(TYPES[dtype])


def values(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


class Pages:
    """A pool, tables and lengths for sequences with n[b] new tokens and
    lens[b] (or lens[b][h]) rows in all.  Pages lie scattered, rows that no
    sequence holds are NaN, table entries behind the last row are -1."""

    def __init__(self, rng, dtype, n, lens, H, D, page, head_pages, extra_width=0):
        self.dtype, self.H, self.D, self.page, self.head = dtype, H, D, page, head_pages
        B = len(n)
        self.lens = np.asarray(lens, dtype=np.int32).reshape(B, H) if head_pages else np.asarray(lens, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        lists = self.lens.reshape(B, -1)
        need = -(-lists // page)
        width = max(1, int(need.max(initial=0))) + extra_width
        total = int(need.sum()) + 2
        ids = rng.permutation(total)
        self.table = np.full((B, lists.shape[1], width), -1, dtype=np.int32)
        at = 0
        shape = (total, page, D) if head_pages else (total, H, page, D)
        self.k = torch.full(shape, float("nan"), dtype=TYPES[dtype])
        self.v = torch.full(shape, float("nan"), dtype=TYPES[dtype])
        for b in range(B):
            for t in range(lists.shape[1]):
                for i in range(need[b, t]):
                    page_id = int(ids[at])
                    at += 1
                    self.table[b, t, i] = page_id
                    rows = min(page, int(lists[b, t]) - i * page)
                    sub = (rows, D) if head_pages else (H, rows, D)
                    for pool in (self.k, self.v):
                        pool[page_id, ..., :rows, :] = rounded(rng.standard_normal(sub), dtype)
        if not head_pages:
            self.table = self.table[:, 0]

    def cuda(self):
        d = {"k_pages": self.k, "v_pages": self.v, "page_table": torch.from_numpy(self.table.copy()),
             "cache_len": torch.from_numpy(self.lens.copy()), "cu_tokens": torch.from_numpy(self.cu.copy())}
        return {k: t.contiguous().cuda() for k, t in d.items()}


def rope_table(n, dim, seed=0):
    """fp32 [n][2][dim / 2] of unit pairs."""
    a = np.random.default_rng(seed).uniform(0, 2 * np.pi, size=(n, dim // 2))
    return np.stack([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def norm_bound(y, mag, dtype, D):
    """How far a stored value of norm_rotate may be off.  One rounding to the
    type (half a step, or half the smallest step).  Before it, in fp32: the
    sum of D squares and its shuffles round at most log2-deep 8 + 4 times
    (relative 12 U32, halved by the root), the mean, eps, root and reciprocal
    5 more, scale, weight and the two products and sum of the rotation 5: at
    most 20 U32 of |a cos| + |b sin|."""
    return HALF[dtype] * (np.abs(y) + 20 * U32 * mag) + 20 * U32 * mag + (FP16_TINY if dtype == "fp16" else 0.0)


def attention_bounds(out, lse, mean_abs, logit_abs, keys, dtype, D):
    """(bound of out, bound of lse).  fp32 errors of a logit: D products
    summed, scaled, shifted by the maximum: at most (D + 6) U32 of logit_abs
    (the shift is a difference of two such logits), and 2^-21 of the result for
    the two approximations of exp2 (2^-22 each; the second is the join's): a
    relative error e of every probability.  Sums of `keys` probabilities in
    fp32 are blocked, at most 2 sqrt(keys) + 32 roundings deep here (slices of
    16, 8 warps, shares).  Then lse is off by e + depth U32 plus its own
    rounding; out by 2 e + 2 depth U32 (numerator and denominator) and half a
    step of the type of the probabilities, all relative to the weighted mean
    of |v|, and by half a step of its own.  fp16 probabilities below 2^-14 have
    a fixed step: at most FP16_TINY each, against a sum of at least 1."""
    e = 2 * (D + 6) * U32 * logit_abs + 2.0 ** -21
    depth = 2 * np.sqrt(keys) + 32
    rel = 2 * e + 2 * depth * U32 + HALF[dtype]
    tiny = FP16_TINY if dtype == "fp16" else 0.0
    vmax = 6.0 * keys * tiny
    b_out = rel[..., None] * mean_abs * (1 + HALF[dtype]) + HALF[dtype] * np.abs(out) + vmax + tiny
    with np.errstate(invalid="ignore"):
        b_lse = e + depth * U32 + 4 * U32 * np.where(np.isfinite(lse), np.abs(lse) + logit_abs, 0.0) + 2.0 ** -22
    return b_out, b_lse
