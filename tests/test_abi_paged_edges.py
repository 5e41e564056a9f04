"""More refusals of the serving calls, before any device work: sizes whose
products pass 64 bits, outputs whose rows lie over one another, and calls that
have nothing to do."""
import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from tests.test_abi_paged import NO_DEVICE, append, attention, norm_rope, strides

no_launch = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: only where nothing can launch")


@no_launch
def test_sizes_whose_products_pass_64_bits():
    for n in (1 << 58, 1 << 61, (1 << 63) - 1):
        assert attention(n=n) == -2
        with pytest.raises(vark.VarkError):
            vark.vark_paged_attention_workspace(n, 2, 64, 8, 128, 16, 3)
    assert attention(n=(1 << 30) // 8) == -2 and attention(n=(1 << 30) // 8 - 1) in NO_DEVICE
    with pytest.raises(vark.VarkError):
        vark.vark_paged_attention_workspace(4, 1 << 23, 8, 4, 128, 16, 3)


@no_launch
def test_outputs_whose_rows_lie_over_one_another():
    assert attention(os=strides(0, 128)) == -3 and attention(os=strides(512, 64)) == -3
    assert attention(qs=strides(0, 0)) in NO_DEVICE                       # rows that are read may
    assert norm_rope(qos=strides(4096, 0, 128)) == -3 and norm_rope(kos=strides(4096, 512, 64)) == -3
    assert norm_rope(qs=strides(4096, 1024, 128)) == -1                   # over itself, by other strides
    assert norm_rope(qs=strides(8, 512, 128)) in NO_DEVICE                # (an axis of one entry)


@no_launch
def test_subnormal_eps_of_unit_length():
    assert norm_rope(norm=2, eps=1e-39) == -1 and append(norm=2, eps=1e-39) == -1
    for norm, eps in ((2, 0.0), (2, 1e-12), (1, 0.0), (1, 1e-39), (0, 1e-39)):
        assert norm_rope(norm=norm, eps=eps) in NO_DEVICE


@no_launch
def test_calls_with_nothing_to_do_need_no_tensors():
    none = dict(q=None, k=None, qo=None, ko=None, pos=None)
    assert norm_rope(T=0, **none) in NO_DEVICE and norm_rope(B=0, **none) in NO_DEVICE
    assert norm_rope(T=0, D=96, **none) == -2 and norm_rope(T=0, norm=5, **none) == -1
    none = dict(k=None, v=None, pos=None)
    assert append(n=0, **none) in NO_DEVICE and append(B=0, table=None, lens=None) in NO_DEVICE
    assert append(n=0, page=24, **none) == -2
    none = dict(q=None, out=None, lse=None)
    assert attention(n=0, **none) in NO_DEVICE and attention(B=0, table=None, lens=None) in NO_DEVICE
    assert attention(n=0, Hq=6, **none) == -2 and attention(n=0, st=None, **none) == -1


def test_binding_strides_of_written_rows():
    bf = torch.bfloat16
    x = torch.zeros(4, 6, 8, 64, dtype=bf)
    for t, fits in ((x[:, :, 2:5], True), (x.transpose(1, 2), True), (x[:1].expand(4, 6, 8, 64), False),
                    (torch.as_strided(x, (2, 3, 2, 64), (192, 64, 128, 1)), False),
                    (torch.as_strided(x, (2, 3, 2, 64), (384, 64, 192, 1)), True),
                    (torch.as_strided(x, (1, 3, 2, 64), (0, 128, 64, 1)), True),
                    (x[..., ::2][..., :32], False)):
        assert vark._strides_fit(t, 2) == fits, (t.shape, t.stride())
    assert vark._strides_fit(x[:1].expand(4, 6, 8, 64), 1)
