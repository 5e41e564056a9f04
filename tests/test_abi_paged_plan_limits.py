"""Sizes at which offsets that go up and down would make the sums of the
attention's plan pass 64 bits are refused on the host; the largest single
sequence is not."""
import pytest
import torch

from tests.test_abi_paged import NO_DEVICE, attention

no_launch = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: only where nothing can launch")

MOST_PAGES = (2 ** 31 - 2048) // 256


def plan_units(n, B, Hq, H, max_rows):
    """The plan's total for offsets 0, n, 0, n, ...: all tokens in every other
    sequence, 16-row tiles, each as heavy as its cache is long."""
    return (B + 1) // 2 * (n * Hq // 16) * 16 * (256 + max_rows)


@no_launch
def test_sums_that_would_pass_64_bits():
    big = dict(page=256, max_pages=MOST_PAGES)
    for n, B, Hq in ((1 << 21, 1 << 14, 8), (1 << 24, 64, 32), (1 << 16, 1 << 20, 8), ((1 << 27) - 1, 16, 8)):
        assert plan_units(n, B, Hq, 4, MOST_PAGES * 256) >= 2 ** 63
        assert attention(n=n, B=B, Hq=Hq, **big) == -2, (n, B, Hq)
    for n, B, Hq in (((1 << 27) - 1, 1, 8), ((1 << 27) - 1, 2, 8), (64, 1 << 20, 8), (1 << 14, 256, 64)):
        assert plan_units(n, B, Hq, 4, MOST_PAGES * 256) < 2 ** 62
        assert attention(n=n, B=B, Hq=Hq, **big) in NO_DEVICE, (n, B, Hq)
    assert attention(n=1 << 17, B=1 << 13, Hq=64, page=256, max_pages=1 << 12) in NO_DEVICE      # caches of 2^20 rows
