"""Compaction whose new lengths are written where the table of pages lies."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_cache_moves import i32, made, raw, tensors
from test_gpu_tree_attention import FMTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 7, 3000])
@pytest.mark.parametrize("pdl", [False, True])
def test_new_lengths_in_the_table(fmt, n, pdl):
    """Every sequence reads its pages before any length is written over them, those of later CTAs too."""
    rng = np.random.default_rng(n)
    wide, page = 3, 16
    table = i32(rng.permutation(n * wide).reshape(n, wide))
    ctx = i32(rng.integers(0, 30, n))
    count = rng.integers(1, 7, n)
    path = i32([[0] + sorted(rng.choice(np.arange(1, 12), k - 1, replace=False).tolist()) + [-1] * (8 - k) for k in count])
    count = i32(count)
    a, b = (made(fmt, 64, 2, page, n * wide, 3) for _ in range(2))
    want = bqg.kv_compact(a, table, ctx, path, count)
    assert torch.equal(want, ctx + count)
    bqg.set_pdl(pdl)
    try:
        for at in (0, n * wide - n, (n * wide - n) // 2):
            for old, t in zip(tensors(made(fmt, 64, 2, page, n * wide, 3)), tensors(b)):
                t.copy_(old)
            over = table.clone()
            out = over.view(-1)[at:at + n]
            assert bqg.kv_compact(b, over, ctx, path, count, out=out) is out
            assert all(torch.equal(raw(x), raw(y)) for x, y in zip(tensors(a), tensors(b)))
            left = table.clone().view(-1)
            left[at:at + n] = want
            assert torch.equal(over.view(-1), left)
            assert bqg.last_device_error() == 0
    finally:
        bqg.set_pdl(False)
