"""The serving calls at values and sizes where a kernel can lose what the
definition keeps: NaN and infinities in a norm's rows."""
import numpy as np
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from oracle import paged as ref
from tests.helpers import check_status, status_word
from tests.paged_cases import Pages, norm_bound, rounded, values
from tests.test_gpu_paged import same_bits

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
