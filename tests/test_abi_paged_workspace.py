"""A workspace asked for once serves every smaller batch: a server keeps one of
its largest shapes."""
import random

import pytest
import torch

import kv_cache_compression_cas_b200 as vark
from tests.test_abi_paged import NO_DEVICE, attention

no_launch = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: only where nothing can launch")


@no_launch
def test_a_workspace_serves_fewer_tokens_and_sequences():
    rng = random.Random(1)
    for _ in range(300):
        H, G, D = rng.choice([1, 2, 8]), rng.choice([1, 2, 4, 5, 40]), rng.choice([64, 128])
        B, n = rng.randint(1, 300), rng.randint(1, 900)
        size = vark.vark_paged_attention_workspace(n, B, H * G, H, D, 16, 3)
        assert 0 < size <= 40 << 20
        for b, m in ((B, n), (1, n), (rng.randint(1, B), rng.randint(1, n)), (rng.randint(1, B), 1)):
            assert attention(n=m, B=b, Hq=H * G, H=H, D=D, ws_bytes=size) in NO_DEVICE, (n, B, m, b, H, G, D)
            assert vark.vark_paged_attention_workspace(m, b, H * G, H, D, 16, 3) <= size
    assert attention(n=64, B=1, ws_bytes=vark.vark_paged_attention_workspace(64, 64, 8, 4, 128, 16, 3)) in NO_DEVICE
    # and what a call refuses is less than its shapes need
    assert attention(n=64, B=1, ws_bytes=vark.vark_paged_attention_workspace(64, 1, 8, 4, 128, 16, 3) - 1) == -1
