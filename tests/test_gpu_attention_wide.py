"""Attention with head_dim 256 and many rows, whose tiles and streams differ from the other widths'."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from test_gpu_tree_attention import FMTS, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,group,page", [(17, 1, 16), (5, 4, 32), (40, 4, 64), (64, 8, 128)])
def test_rows_and_pages(fmt, T, group, page):
    Case(fmt, 256, 2, group, [0, 131, 1000], [T, 1, T], page=page, tree=True, seed=T).check()


@pytest.mark.parametrize("fmt", FMTS)
def test_long_context_is_split(fmt):
    """One sequence over every CTA: joined partial results, the same bits each time."""
    c = Case(fmt, 256, 1, 4, [20000], [40], page=64, tree=True, seed=5)
    a = c.run()
    c.check(a)
    for _ in range(3):
        assert torch.equal(a.view(torch.int16), c.run().view(torch.int16))
    assert not c.ws[:4096 * 4].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_many_pieces_per_cta(fmt):
    rng = np.random.default_rng(8)
    ctx, new = rng.integers(0, 300, 120).tolist(), rng.integers(0, 10, 120).tolist()
    Case(fmt, 256, 2, 4, ctx, new + [], page=16, tree=True, seed=10).check()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_see_nothing_and_masked_infinities(fmt):
    T = 30
    for value in (float("nan"), float("inf")):
        c = Case(fmt, 256, 2, 2, [0, 37], [T, T], tree=True, seed=6)
        c.mask[0] = 0
        hit = 2
        words = [int(w) & (2 ** 64 - 1) for w in c.mask.tolist()][T:]
        clear = [T + i for i, w in enumerate(words) if not (w >> hit) & 1]
        seen = [T + i for i, w in enumerate(words) if (w >> hit) & 1]
        c.spoil(1, 37 + hit, value, "v")
        got = c.run()
        assert not got[0].any()
        out, *sizes = ref.attention(c.q, c.cache, c.table, c.ctx, c.start, c.mask, c.scale)
        bound = ref.attention_bound(fmt, 256, out, *sizes)[clear]
        assert ((got.double().cpu()[clear] - out[clear]).abs() <= bound).all()
        assert not torch.isfinite(got[seen]).all(-1).any()


@pytest.mark.parametrize("fmt", FMTS)
def test_missing_pages_are_not_seen(fmt):
    """A page index outside the cache: its tokens count for no row, and the call says so."""
    c = Case(fmt, 256, 2, 4, [300], [20], page=32, seed=3, junk=False)
    c.table[0, 4] = -1
    got = c.run().double().cpu()
    assert bqg.last_device_error() == bqg.DEVERR_PAGE
    keep = [p for i, p in enumerate(c.table[0].tolist()) if i != 4]
    c.table = torch.tensor([keep], dtype=torch.int32, device="cuda")
    c.ctx = c.ctx - 32
    out, *sizes = ref.attention(c.q, c.cache, c.table, c.ctx, c.start, c.mask, c.scale)
    assert ((got - out).abs() <= ref.attention_bound(fmt, 256, out, *sizes)).all()
