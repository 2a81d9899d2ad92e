"""Attention behind shared prefixes, against fp64 over each sequence's whole context."""
import math

import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_attention_edges import bound, reference
from test_gpu_tree_attention import FMTS, fill, tree_words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


class Shared:
    """Groups of sequences: prefix[g] tokens shared by per[g] of them; own[i] and new[i] tokens of sequence i.  The first
    of a group holds the prefix; the others' rows have no pages for it, and what their copy of the page where it ends
    holds of it is no number.  `full`: the block table in which each sequence has it all, for the reference."""

    def __init__(self, fmt, D, n_kv, group, prefix, per, own, new, page=16, tree=False, seed=0, spread=1.0, spoil=True):
        rng = np.random.default_rng(seed)
        n, P = sum(per), page
        head = [p for p, k in zip(prefix, per) for _ in range(k)]
        first = np.concatenate([[0], np.cumsum(per)])
        ctx = [h + o for h, o in zip(head, own)]
        wide = max((c + t + P - 1) // P for c, t in zip(ctx, new)) + 1
        self.cache = bqg.kv_cache(fmt, n * wide + n + 1, n_kv, P, D)
        fill(self.cache, seed, spread)
        order = rng.permutation(n * wide)
        table = order.reshape(n, wide).astype(np.int32)
        for g, k in enumerate(per):
            for i in range(first[g], first[g + 1]):
                table[i, :prefix[g] // P] = table[first[g], :prefix[g] // P]
        self.first = first
        dev = lambda a, t=torch.int32: torch.tensor(np.asarray(a), dtype=t, device="cuda")
        self.table, self.ctx, self.prefix, self.seqs = dev(table), dev(ctx), dev(prefix), dev(first)
        self.start = dev(np.concatenate([[0], np.cumsum(new)]))
        self.n, self.H, self.max_q = sum(new), n_kv * group, max(max(new), 1)
        self.most = max(max(sum(new[first[g]:first[g + 1]]) for g in range(len(per))), 1)
        self.q = (torch.randn(self.n, self.H, D, generator=torch.Generator().manual_seed(seed + 1)) * 1.5).to(torch.bfloat16).cuda()
        self.mask = tree_words(rng, new).cuda() if tree else None
        self.scale = 1 / math.sqrt(D)
        tensors = [t for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale) if t is not None]
        for g, p in enumerate(prefix):                      # the page where a prefix ends: the same tokens in all copies
            if p % P:
                for i in range(first[g] + 1, first[g + 1]):
                    for t in tensors:
                        t[int(table[i, p // P]), :, :p % P] = t[int(table[first[g], p // P]), :, :p % P]
        for b, (c, t) in enumerate(zip(ctx, new)):          # what lies behind each sequence's end is no number
            for at in range(c + t, wide * P):
                self.nan(b, at)
        self.want = reference(self)
        # rows of a pass are at most max_q or `most` x group: the keys' rounding to fp16 counts for either
        self.limit_rows = max(self.max_q, self.most)
        keep, self.max_q = self.max_q, self.limit_rows
        self.limit = bound(self, *self.want)
        self.max_q = keep
        self.full = self.table.clone()
        if spoil:
            for g, p in enumerate(prefix):
                for i in range(first[g] + 1, first[g + 1]):
                    self.table[i, :p // P] = -1
                    for at in range(p // P * P, p):
                        self.nan(i, at)
        self.ws = bqg.shared_prefix_attention_workspace(self.cache, self.H, n, self.max_q, self.n, len(prefix),
                                                        max_shared=self.most)

    def nan(self, b, at):
        P, c = self.cache.page_size, self.cache
        page = int(self.table[b, at // P])
        for t in ((c.k, c.v) if c.fmt == bqg.BF16 else (c.k_scale, c.v_scale)):
            t[page, :, at % P] = float("nan")

    def run(self, **kw):
        a = dict(mask=self.mask, max_shared=self.most, scale=self.scale, ws=self.ws, seq_start=self.seqs)
        a.update(kw)
        return bqg.shared_prefix_attention(a.pop("q", self.q), self.cache, self.table, self.ctx, self.start, self.max_q,
                                           self.prefix, **a)

    def check(self, got=None, rows=slice(None)):
        got = (self.run() if got is None else got).double()[rows]
        assert torch.isfinite(got).all()
        want, limit = self.want[0][rows], self.limit[rows]
        assert ((got - want).abs() <= limit).all(), ((got - want).abs() / limit).max().item()
        assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("per,group", [(1, 1), (2, 4), (3, 5), (16, 1), (20, 4), (33, 8)])
@pytest.mark.parametrize("prefix", [1, 16, 63, 64, 130])
def test_one_token_each(fmt, D, per, group, prefix):
    own = [(7 * i) % 50 for i in range(per)]
    Shared(fmt, D, 2, group, [prefix], [per], own, [1] * per, seed=prefix + D).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group,per", [(2, 4, 2), (5, 3, 1), (9, 8, 3), (33, 4, 2), (64, 1, 3)])
@pytest.mark.parametrize("tree", [False, True])
def test_new_tokens(fmt, D, T, group, per, tree):
    own = [70, 0, 200][:per]
    new = [T, 1, max(1, T - 3)][:per]
    Shared(fmt, D, 2, group, [93], [per], own, new, tree=tree, seed=T + D, page=32).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_several_prefixes(fmt, D, page):
    """Ragged everything: a prefix of no tokens, one of a single sequence, one without sequences, sequences without new tokens."""
    prefix, per = [300, 0, 17, 128, 40], [4, 3, 1, 0, 5]
    own = [0, 10, 129, 700, 5, 0, 64, 1, 30, 0, 0, 300, 2]
    new = [1, 3, 0, 20, 1, 2, 0, 4, 0, 1, 64, 7, 1]
    Shared(fmt, D, 3, 2, prefix, per, own, new, page=page, tree=True, seed=page).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("per,T,group", [(2, 1, 4), (12, 1, 4), (64, 1, 4), (5, 13, 4), (30, 8, 8)])
def test_a_long_prefix_is_split(fmt, per, T, group):
    """One prefix over every CTA, twice the same bits, the counters back at zero."""
    c = Shared(fmt, 128, 1, group, [20000], [per], [30] * per, [T] * per, page=64, tree=T > 1, seed=T)
    a = c.run()
    c.check(a)
    for _ in range(3):
        assert torch.equal(a.view(torch.int16), c.run().view(torch.int16))
    assert not c.ws[:4096 * 4].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences_and_prefixes(fmt):
    rng = np.random.default_rng(4)
    per = rng.integers(0, 9, 40).tolist()
    n = sum(per)
    Shared(fmt, 128, 2, 2, rng.integers(0, 90, 40).tolist(), per, rng.integers(0, 40, n).tolist(),
           rng.integers(0, 4, n).tolist(), seed=9).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 20])
def test_nothing_shared_is_tree_attention(fmt, T):
    """A prefix of no tokens: the own pass alone.  Many rows go to the ordinary call's kernel: the same bits."""
    c = Shared(fmt, 128, 2, 4, [0], [3], [100, 40, 0], [T, 1, T], page=32, tree=True, seed=3)
    ws = bqg.tree_attention_workspace(c.cache, c.H, 3, c.max_q)
    plain = bqg.tree_attention(c.q, c.cache, c.table, c.ctx, c.start, c.max_q, mask=c.mask, scale=c.scale, ws=ws)
    c.check()
    c.check(plain)
    if T == 20:
        assert torch.equal(c.run().view(torch.int16), plain.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [4, 30])
def test_rows_that_see_nothing(fmt, T):
    """No new token seen and no own context: the prefix alone, and without one zeros."""
    c = Shared(fmt, 128, 2, 4, [50, 0], [2, 1], [0, 30, 0], [T, T, T], tree=True, seed=3)
    c.mask[0] = 0
    c.mask[2 * T] = 0
    c.want = reference_of(c)
    c.check()
    assert not c.run()[2 * T].any() and c.run()[0].any()


def reference_of(c):
    """The reference again, over the full table (the spoiled copies are put right for it)."""
    keep = c.table, [t.clone() for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale) if t is not None]
    tensors = [t for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale) if t is not None]
    P = c.cache.page_size
    for g, p in enumerate(c.prefix.tolist()):
        for i in range(c.first[g] + 1, c.first[g + 1]):
            for t in tensors:
                t[int(c.full[i, p // P]), :, :p % P] = t[int(c.full[c.first[g], p // P]), :, :p % P]
    c.table = c.full
    out = reference(c)
    c.table = keep[0]
    for t, old in zip(tensors, keep[1]):
        t.copy_(old)
    return out


@pytest.mark.parametrize("fmt", FMTS)
def test_far_scores(fmt):
    """Scores of thousands: one part's maximum is far above the other's."""
    Shared(fmt, 128, 2, 4, [300], [3], [200, 5, 90], [3, 1, 2], seed=11, spread=20.0).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [3, 30])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_shared_infinity_or_nan_reaches_its_sequences_alone(fmt, T, value):
    c = Shared(fmt, 128, 2, 4, [45, 45], [2, 2], [10, 20, 0, 3], [T, 1, T, 1], seed=5)
    page = int(c.full[0, 2])                                # tokens 32 .. 47 of the first group
    t = c.cache.v if fmt == bqg.BF16 else c.cache.v_scale
    t[page, :, 5] = value
    got = c.run()
    assert not torch.isfinite(got[:T + 1]).all(-1).any()
    c.check(got, slice(T + 1, None))


def test_strided_queries_streams_and_graphs():
    c = Shared(bqg.Q8_0, 128, 2, 4, [200, 33], [6, 2], [20] * 8, [3, 1] * 4, page=32, seed=13)
    wide = torch.full((c.n, c.H * 128 + 64), 9.0, dtype=torch.bfloat16, device="cuda")
    part = wide[:, :c.H * 128].unflatten(-1, (c.H, 128))
    part.copy_(c.q)
    want = c.run()
    c.check(want)
    assert torch.equal(c.run(q=part), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out)
    for pdl in (False, True):
        bqg.set_pdl(pdl)
        try:
            out.fill_(7)
            g.replay()
            assert torch.equal(out, want)
            assert torch.equal(c.run(), want)
        finally:
            bqg.set_pdl(False)


def test_one_prefix_without_offsets_and_default_sizes():
    c = Shared(bqg.BF16, 128, 2, 4, [100], [3], [20, 0, 5], [2, 1, 1], seed=8)
    want = c.run()
    ws = bqg.shared_prefix_attention_workspace(c.cache, c.H, 5, 7, 40)
    assert torch.equal(c.run(seq_start=None, max_shared=None, ws=ws), want)
    c.check(want)


def test_one_workspace_for_calls_of_different_shapes():
    big = Shared(bqg.BF16, 256, 2, 4, [500], [9], [30] * 9, [30] * 9, page=64, seed=1)
    small = [Shared(f, D, 2, g, [300, 20], [2, 3], [9] * 5, [t] * 5, page=64, seed=2)
             for f in FMTS for D, g, t in ((64, 1, 1), (128, 8, 9), (256, 2, 3))]
    ws = torch.zeros(max(c.ws.numel() for c in [big, *small]), dtype=torch.uint8, device="cuda")
    for c in [big, *small, big]:
        c.ws = ws
        c.check()


def test_bad_lengths_are_reported():
    c = Shared(bqg.Q8_0, 128, 2, 2, [40, 60], [2, 2], [10, 20, 0, 3], [2, 1, 1, 2], page=16, seed=5, spoil=False)
    c.check()
    # more query tokens than said: the prefix counts as not shared
    got = c.run(max_shared=2)
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH
    c.check(got)
    keep = c.prefix.clone()
    for bad in ([-3, 60], [10 ** 9, 60], [45, 61]):          # below 0; beyond the pages; beyond a context (60 + 0)
        c.prefix.copy_(torch.tensor(bad, dtype=torch.int32))
        c.run()
        assert bqg.last_device_error() == bqg.DEVERR_LENGTH
    c.prefix.copy_(keep)
    seqs = c.seqs.clone()
    for bad in ([0, 2, 3], [1, 2, 4], [0, 9, 4], [0, -1, 4], [4, 2, 0]):
        c.seqs.copy_(torch.tensor(bad, dtype=torch.int32))
        c.run()
        assert bqg.last_device_error() == bqg.DEVERR_LENGTH
    c.seqs.copy_(torch.tensor([0, 0, 4], dtype=torch.int32))  # all four behind the second prefix: longer than two contexts
    c.run()
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH
    c.seqs.copy_(seqs)
    c.table[0, 1] = -1                                       # tokens 16 .. 31 of the first prefix
    c.run()
    assert bqg.last_device_error() == bqg.DEVERR_PAGE


def test_workspace_is_required():
    c = Shared(bqg.BF16, 64, 1, 1, [5], [2], [5, 6], [1, 1])
    for ws in (None, c.ws[:-16]):
        with pytest.raises(bqg.BqgError) as e:
            c.run(ws=ws)
        assert e.value.status == 7
    with pytest.raises(ValueError):
        c.prefix = torch.zeros(2, dtype=torch.int32, device="cuda")
        c.run(seq_start=None)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 9])
def test_pages_beyond_32_bits_of_bytes(fmt, T):
    """The same pages at the end of a cache of more than 2^32 bytes a side: the same bits."""
    small = Shared(fmt, 128, 2, 4, [100], [3], [40, 0, 70], [T, 1, T], page=64, seed=4)
    want = small.run()
    row = 2 * 64 * (256 if fmt == bqg.BF16 else 128 if fmt == bqg.Q8_0 else 64)
    old = small.cache
    shift = 2 ** 32 // row + 1
    small.cache = bqg.kv_cache(fmt, shift + old.n_pages, 2, 64, 128)
    for name in ("k", "v", "k_scale", "v_scale"):
        if getattr(old, name) is not None:
            getattr(small.cache, name)[shift:] = getattr(old, name)
    small.table = torch.where(small.table < 0, small.table, small.table + shift)
    assert torch.equal(small.run().view(torch.int16), want.view(torch.int16))
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_calls_in_turn_on_one_workspace_leave_nothing_behind(fmt):
    """Two captured calls of different sequences on one workspace, replayed in turns, with and without a prefix."""
    a = Shared(fmt, 128, 2, 4, [300], [5], [30, 0, 70, 9, 1], [2, 1, 4, 1, 1], page=32, seed=4)
    b = Shared(fmt, 128, 2, 4, [0, 50], [2, 3], [200, 0, 70, 9, 1], [1, 1, 30, 1, 3], page=32, seed=5)
    ws = torch.zeros(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        c.ws = ws
        out = torch.zeros_like(c.q)
        c.run(out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out)
        graphs.append((c, g, out, c.run()))
    for _ in range(3):
        for c, g, out, want in graphs:
            out.fill_(7)
            g.replay()
            assert torch.equal(out, want)
            c.check(out)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_workspace_for_more_serves_fewer(fmt, D):
    cache = bqg.kv_cache(fmt, 1, 1, 16, D)
    size = lambda group, q, n, most: bqg.shared_prefix_attention_workspace(cache, group, 64, q, n, 1, max_shared=most).numel()
    for group in (1, 2, 3, 5, 8, 16, 64):
        for sizes in ([size(group, q, 64, 64) for q in range(1, 65)], [size(group, 1, 64, m) for m in range(0, 65)],
                      [size(group, 3, n, 64) for n in range(1, 130)]):
            assert sizes == sorted(sizes), (group, sizes)
