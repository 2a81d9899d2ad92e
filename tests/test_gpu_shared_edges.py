"""Attention behind shared prefixes where lengths do not fit, and where a page's unneeded places hold no numbers."""
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_shared_prefix import Shared
from test_gpu_tree_attention import FMTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("page", [16, 128])
def test_a_prefix_that_does_not_fit_is_not_shared(fmt, D, T, page):
    """As long as the row of the table or longer, or below zero: every row is written, and is the one without sharing."""
    c = Shared(fmt, D, 2, 3, [40, 60], [2, 2], [10, 20, 0, 3], [T, 1, T, 1], page=page, seed=5, spoil=False)
    whole = c.table.shape[1] * page
    keep = c.prefix.clone()
    for bad in (whole, whole + 1, 10 ** 9, 2 ** 31 - 1, -1, -2 ** 31):
        for g in (0, 1):
            c.prefix.copy_(keep)
            c.prefix[g] = bad
            out = torch.full_like(c.q, float("nan"))
            c.run(out=out)
            assert bqg.last_device_error() == bqg.DEVERR_LENGTH
            c.check(out)
    # the longest that is shared: nothing of the first two contexts is right, but their rows are written too
    c.prefix.copy_(keep)
    c.prefix[0] = whole - 1
    out = torch.full_like(c.q, 12345.0)
    c.run(out=out)
    assert bqg.last_device_error() & bqg.DEVERR_LENGTH
    assert not (out == 12345.0).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 20])
def test_a_prefix_that_fills_the_table_of_sequences_without_new_tokens(fmt, T):
    """Nothing is to be computed there, and nothing is wrong."""
    c = Shared(fmt, 128, 2, 2, [32, 7], [2, 1], [0, 0, 2], [0, 0, T], page=16, seed=6, spoil=False)
    c.prefix[0] = c.ctx[0] = c.ctx[1] = c.table.shape[1] * 16
    c.check()


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("length", [10 ** 6, 2 ** 31 - 1, -1])
def test_a_prefix_without_sequences_may_have_any_length(T, length):
    """It is nobody's, so nothing does not fit."""
    c = Shared(bqg.Q8_0, 128, 2, 2, [32, 9, 7], [2, 0, 1], [5, 0, 2], [T, 0, T], page=16, seed=6)
    c.prefix[1] = length
    c.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group", [(1, 1), (2, 4), (9, 4), (20, 5)])
def test_places_of_the_prefix_in_other_pages_change_nothing(fmt, D, T, group):
    """What a sequence's own page holds in the shared tokens' places, numbers or none, does not show in a single bit."""
    make = lambda spoil: Shared(fmt, D, 2, group, [45, 70], [3, 2], [10, 300, 0, 3, 40], [T, 1, T, 1, T], page=32, seed=7, spoil=spoil)
    a, b = make(False), make(True)
    assert torch.equal(a.run().view(torch.int16), b.run().view(torch.int16))
    b.check()
