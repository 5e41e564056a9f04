"""The serving calls at values and sizes where a kernel can lose what the
definition keeps: NaN and infinities in a norm's rows; caches where one key
outweighs the others; temperatures next to 0."""
import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from oracle import paged as ref
from tests.helpers import check_status, status_word
from tests.paged_cases import FP16_TINY, HALF, U32, Pages, attention_bounds, norm_bound, rounded, values
from tests.test_gpu_paged import compare, run_attention, same_bits

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("norm", [vark.VARK_NORM_RMS, vark.VARK_NORM_L2])
def test_nan_and_infinity_in_a_normed_row(dtype, D, norm):
    """A NaN anywhere in a row makes its norm, and so the whole row, NaN; an
    infinity its own channel NaN and the others 0; the rows beside them are
    what they were."""
    rng = np.random.default_rng(D + norm)
    B, T, H, eps = 1, 6, 5, 1e-6
    x = rounded(rng.standard_normal((B, T, H, D)), dtype)
    x[0, 1, 2, 7] = float("nan")
    x[0, 2, 0, D - 1] = float("nan")
    x[0, 3, 4, 20] = float("inf")
    x[0, 4, 1, 0] = -float("inf")
    st = status_word()
    got = torch.zeros(B, T, H, D, dtype=x.dtype, device="cuda")
    vark.vark_qk_norm_rope(x.cuda(), None, got, None, norm, None, None, eps, None, None, st)
    check_status(st)
    with np.errstate(invalid="ignore"):
        y, mag = ref.norm_rotate(values(x)[0], norm, None, eps, None, None, False)
    assert np.isnan(y[1, 2]).all() and np.isnan(y[2, 0]).all()
    g = values(got)[0]
    assert (np.isnan(g) == np.isnan(y)).all()
    live = ~np.isnan(y)
    assert (np.abs(g - y)[live] <= norm_bound(y, mag, dtype, D)[live]).all()
    # the append's keys are the same rows
    pg = Pages(rng, dtype, [T], [T], H, D, 16, False)
    d = pg.cuda()
    vark.vark_paged_append(x[0].cuda(), x[0].cuda(), d["cu_tokens"], d["k_pages"], d["v_pages"], d["page_table"],
                           d["cache_len"], norm, None, eps, None, None, st)
    check_status(st)
    page = int(pg.table[0, 0])
    assert (np.isnan(values(d["k_pages"][page, :, :T])) == np.isnan(y).transpose(1, 0, 2)).all()
    keys = torch.nan_to_num(d["k_pages"][page, :, :T].transpose(0, 1), nan=1.0)
    assert same_bits(keys, torch.nan_to_num(got[0], nan=1.0))


# ------------------------------------------------------------------ attention
def mma_sum_loss(keys, tiles):
    """What sums on the tensor cores lose, of the mean of |v|: an MMA adds 16
    products to an fp32 sum after cutting them off 2^-25 below its leading bit,
    then cuts the sum to 24 bits: 16 * 2^-25 + 2^-23 = 20 * 2^-25 for 16 keys.  A
    sum takes at most 256 * 128 keys on tcgen05, an eighth of the keys (a warp's)
    in the kernels of few rows."""
    return (min(keys, 256 * 128) if tiles else keys / 8) * 1.25 * 2.0 ** -25


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap", [17.0, 18.0, 10.0])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 20), (40, 4)])
@pytest.mark.parametrize("value", [0.0, None])
def test_one_key_outweighs_a_long_cache(dtype, D, gap, n, G, value):
    """The first of 65536 keys has a logit `gap` above the others, which are
    alike and whose weights together are felt all the same; its value is 0, so
    the others make all of the output, or as theirs, so that each adds next to
    nothing to a large sum.  160 sequences over the same pages, so
    that a CTA has long runs of keys (one is half a cache and more); every
    kernel: 16, 32 and 256 rows."""
    rng = np.random.default_rng(int(gap) * 1000 + D + G)
    B, keys, ps = 160, 65536, 256
    k = np.zeros((keys // ps, 1, ps, D))
    k[0, 0, 0] = np.float16(gap / np.sqrt(D))           # with q = 1: D of them / sqrt(D)
    k = rounded(k, dtype)
    v = rounded(rng.uniform(0.5, 1.5, (keys // ps, 1, ps, D)), dtype)
    if value is not None:
        v[0, 0, 0] = value
    table = np.arange(keys // ps, dtype=np.int32)[None]
    lens, cu = np.array([keys], dtype=np.int32), np.array([0, 1], dtype=np.int32)
    one = np.ones((1, 1, D))
    o, z, mean_abs, logit_abs = ref.paged_attention(one, cu, values(k), values(v), table, lens, np.ones(1), False)
    N = B * n
    out = torch.empty(N, G, D, dtype=k.dtype, device="cuda")
    lse = torch.empty(N, G, device="cuda")
    ws = torch.empty(vark.vark_paged_attention_workspace(N, B, G, 1, D, ps, keys // ps), dtype=torch.uint8,
                     device="cuda")
    st = status_word()
    vark.vark_paged_attention(torch.ones(N, G, D, dtype=k.dtype, device="cuda"),
                              torch.arange(B + 1, dtype=torch.int32, device="cuda") * n, k.cuda(), v.cuda(),
                              torch.from_numpy(table).cuda().expand(B, keys // ps).contiguous(),
                              torch.from_numpy(lens).cuda().expand(B).contiguous(), None, False, out, lse, ws, st)
    check_status(st)
    b_out, b_lse = attention_bounds(o, z, mean_abs, logit_abs, float(keys), dtype, D)
    if dtype == "fp16":
        # the bound allows every probability FP16_TINY of the largest, times 6 for |v|; the
        # reference 2^7 below the maximum makes it 2^-7 of that, and |v| is at most 1.5
        b_out += keys * FP16_TINY * (1.5 * 2.0 ** -7 - 6.0)
    b_out += mma_sum_loss(keys, n > 1) * mean_abs
    assert (np.abs(values(out) - o[0, 0]) <= b_out[0, 0]).all()
    assert (np.abs(values(lse) - z[0, 0]) <= b_lse[0, 0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 20), (40, 4)])
def test_mean_of_a_million_keys(dtype, D, n, G):
    """Logits all 0 (a temperature of 0): the output is the mean of the values,
    the log-sum the logarithm of their number.  160 sequences over the same
    eight pages, again and again."""
    rng = np.random.default_rng(D + G)
    B, keys, ps = 160, 1 << 20, 256
    v = rounded(rng.uniform(0.5, 1.5, (8, 1, ps, D)), dtype)
    k = rounded(rng.standard_normal((8, 1, ps, D)), dtype)
    want = values(v).reshape(-1, D).mean(0)
    N = B * n
    out = torch.empty(N, G, D, dtype=v.dtype, device="cuda")
    lse = torch.empty(N, G, device="cuda")
    ws = torch.empty(vark.vark_paged_attention_workspace(N, B, G, 1, D, ps, keys // ps), dtype=torch.uint8,
                     device="cuda")
    st = status_word()
    vark.vark_paged_attention(torch.ones(N, G, D, dtype=v.dtype, device="cuda"),
                              torch.arange(B + 1, dtype=torch.int32, device="cuda") * n, k.cuda(), v.cuda(),
                              torch.arange(keys // ps, dtype=torch.int32, device="cuda").remainder(8).expand(B, -1)
                              .contiguous(), torch.full((B,), keys, dtype=torch.int32, device="cuda"),
                              torch.zeros(G, device="cuda"), False, out, lse, ws, st)
    check_status(st)
    # every probability is a power of two and their sum exact; each of 80 partial sums rounds once
    bound = want * (HALF[dtype] + mma_sum_loss(keys, n > 1) + 80 * U32)
    assert (np.abs(values(out) - want) <= bound).all()
    assert (np.abs(values(lse) - np.log(keys)) <= 16 * U32 * np.log(keys)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 90])
def test_temperatures_next_to_zero(dtype, D, n):
    """The smallest temperatures of either sign, some of whose products with
    log2(e) / sqrt(D) are 0 in fp32: masked keys stay masked in every kernel."""
    rng = np.random.default_rng(D + n)
    pg = Pages(rng, dtype, [n, n], [n + 40, n + 300], 1, D, 32, False)
    tau = np.array([1e-45, -1e-45, 3e-45, -4e-45, 1e-44, 1e-38, -1e-30, 0.0], dtype=np.float32)
    q = rounded(rng.standard_normal((2 * n, len(tau), D)), dtype)
    out, lse = run_attention(pg, q, tau, True)
    compare(pg, q, tau, True, out, lse, dtype)
