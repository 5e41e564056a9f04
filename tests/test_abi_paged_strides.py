"""Outputs of vark_qk_norm_rope whose rows share elements are refused by the
library itself, whatever order their axes are in; before any device work."""
import ctypes
import itertools
import random

import pytest
import torch

from tests.test_abi_paged import NO_DEVICE, norm_rope, strides

APART = dict(qo=ctypes.c_void_p(8192), ko=ctypes.c_void_p(12288))        # not written over the inputs

no_launch = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: only where nothing can launch")


@no_launch
@pytest.mark.parametrize("out,heads", [("qos", "Hq"), ("kos", "Hk")])
def test_rows_that_share_elements(out, heads):
    for s in ((4096, 128, 128), (4096, 256, 128), (128, 128, 1024), (2048, 1024, 1000), (0, 1024, 64),
              (1 << 62, 896, 128)):
        assert norm_rope(**{out: strides(*s), heads: 8, "B": 2}, **APART) == -3, s
    for s in ((4096, 1024, 128), (128, 2048, 256), (1024 * 8, 128, 512), (1 << 62, 1024, 128)):
        assert norm_rope(**{out: strides(*s), heads: 8, "B": 2}, **APART) in NO_DEVICE, s
    assert norm_rope(**{out: strides(0, 128, 128), heads: 1}, **APART) in NO_DEVICE      # axes of one entry have no step


@no_launch
def test_against_every_row():
    """Small shapes and strides, by the rows themselves.  (The rule is that of
    nested axes: it may refuse rows that interleave without touching, never
    pass ones that touch.)"""
    rng = random.Random(0)
    passed = 0
    for _ in range(4000):
        B, T, H = (rng.randint(1, 4) for _ in range(3))
        s = [64 * rng.randint(1, 14) for _ in range(3)]
        starts = [b * s[0] + t * s[1] + h * s[2] for b, t, h in itertools.product(range(B), range(T), range(H))]
        starts.sort()
        apart = all(y - x >= 64 for x, y in zip(starts, starts[1:]))
        rc = norm_rope(D=64, B=B, T=T, Hq=H, qos=strides(*s), **APART)
        assert rc in (-3, *NO_DEVICE)
        passed += rc != -3
        assert apart or rc == -3, (B, T, H, s)
    assert passed > 400
