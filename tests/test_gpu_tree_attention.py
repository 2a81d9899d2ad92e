"""Attention of the newest tokens over a paged cache, against fp64 over the
visible tokens alone, within the bound of kv_reference.attention_bound."""
import math

import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from block_quantized_gemv_gb300 import build as bqg_build

pytestmark = pytest.mark.gpu

FMTS = [bqg.BF16, bqg.Q8_0, bqg.Q4_0]


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


def fill(cache, seed, spread=1.0):
    """Random codes and scales (bf16: values) everywhere: about `spread` in size."""
    g = torch.Generator().manual_seed(seed)
    for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if cache.fmt == bqg.BF16:
            codes.copy_((torch.randn(codes.shape, generator=g) * spread).to(torch.bfloat16))
        else:
            lo, hi, step = (-127, 128, 3.0 / 127) if cache.fmt == bqg.Q8_0 else (0, 256, 3.0 / 8)
            codes.copy_(torch.randint(lo, hi, codes.shape, generator=g, dtype=torch.int32).to(codes.dtype))
            scales.copy_((torch.rand(scales.shape, generator=g) * step * spread).to(torch.float16))


def tree_words(rng, lens):
    """Ancestor masks of random trees, one word per new token."""
    out = []
    for T in lens:
        words = []
        for t in range(T):
            parent = int(rng.integers(-1, t))
            words.append((words[parent] if parent >= 0 else 0) | (1 << t))
        out += words
    return torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in out], dtype=torch.int64)


class Case:
    def __init__(self, fmt, D, n_kv, group, ctx, new, page=16, tree=False, seed=0, spread=1.0, junk=True):
        rng = np.random.default_rng(seed)
        per = max((c + t + page - 1) // page for c, t in zip(ctx, new)) + 1
        self.cache = bqg.kv_cache(fmt, len(ctx) * per + 1, n_kv, page, D)
        fill(self.cache, seed, spread)
        self.table = torch.from_numpy(rng.permutation(len(ctx) * per).reshape(len(ctx), per).astype(np.int32)).cuda()
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        self.n, self.H, self.max_q = sum(new), n_kv * group, max(max(new), 1)
        self.q = (torch.randn(self.n, self.H, D, generator=torch.Generator().manual_seed(seed + 1)) * 1.5).to(torch.bfloat16).cuda()
        self.mask = tree_words(rng, new).cuda() if tree else None
        self.scale = 1 / math.sqrt(D)
        if junk:                                            # what lies behind each sequence's end is no number
            for b, (c, t) in enumerate(zip(ctx, new)):
                for at in range(c + t, per * page):
                    self.spoil(b, at)
        self.ws = bqg.tree_attention_workspace(self.cache, self.H, len(ctx), self.max_q)

    def spoil(self, b, at, value=float("nan"), which="kv"):
        P, c = self.cache.page_size, self.cache
        page = int(self.table[b, at // P])
        for name in which:
            t = getattr(c, name) if c.fmt == bqg.BF16 else getattr(c, name + "_scale")
            t[page, :, at % P] = value

    def run(self, **kw):
        kw.setdefault("mask", self.mask)
        return bqg.tree_attention(kw.pop("q", self.q), self.cache, self.table, self.ctx, self.start, self.max_q,
                                  scale=self.scale, ws=self.ws, **kw)

    def check(self, got=None, rows=None):
        got = (self.run() if got is None else got).double().cpu()
        out, *sizes = ref.attention(self.q, self.cache, self.table, self.ctx, self.start, self.mask, self.scale)
        bound = ref.attention_bound(self.cache.fmt, self.cache.head_dim, out, *sizes)
        if rows is not None:
            got, out, bound = got[rows], out[rows], bound[rows]
        assert torch.isfinite(got).all()
        worst = ((got - out).abs() / bound).max().item() if got.numel() else 0.0
        assert worst <= 1, worst
        assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 7])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 63, 64, 65, 500])
def test_one_token(fmt, D, group, ctx):
    Case(fmt, D, 2, group, [ctx], [1], seed=ctx + D).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group", [(2, 4), (5, 3), (16, 1), (17, 1), (9, 8), (33, 4), (64, 1), (64, 5)])
@pytest.mark.parametrize("tree", [False, True])
def test_new_tokens(fmt, D, T, group, tree):
    Case(fmt, D, 2, group, [70], [T], tree=tree, seed=T + D, page=32).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_ragged_batch(fmt, D, page):
    ctx = [0, 300, 17, 1, 0, 129, 64, 1000, 5]
    new = [1, 3, 0, 20, 2, 1, 64, 7, 0]
    Case(fmt, D, 3, 2, ctx, new, page=page, tree=True, seed=page).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,group", [(1, 1), (1, 8), (6, 4), (40, 4)])
def test_long_context_is_split(fmt, T, group):
    """One sequence over every CTA: joined partial results, the same bits each time."""
    c = Case(fmt, 128, 1, group, [30000], [T], page=64, tree=T > 1, seed=T)
    a = c.run()
    c.check(a)
    for _ in range(3):
        assert torch.equal(a.view(torch.int16), c.run().view(torch.int16))
    assert not c.ws[:4096 * 4].any()                        # the counters are back at zero


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences(fmt, D):
    rng = np.random.default_rng(4)
    ctx, new = rng.integers(0, 40, 150).tolist(), rng.integers(0, 3, 150).tolist()
    Case(fmt, D, 2, 2, ctx, new, seed=9).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,group", [(4, 2), (20, 4), (64, 4)])
def test_rows_that_see_nothing_are_zero(fmt, T, group):
    c = Case(fmt, 128, 2, group, [0, 40], [T, T], tree=True, seed=3)
    c.mask[0] = 0                                           # no context and no new token: an empty row
    c.mask[T - 1] = 1 << 1
    c.mask[T + 1] = 0                                       # its context alone
    c.check()
    assert not c.run()[0].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,group", [(5, 2), (30, 2), (64, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_masked_infinity_or_nan_reaches_nobody(fmt, T, group, value):
    """One drafted token's key and value are spoiled: rows that do not see it stay right, rows that do are not finite."""
    for which in ("k", "v", "kv"):
        c = Case(fmt, 128, 2, group, [37], [T], tree=True, seed=6)
        hit = 2
        words = [int(w) & (2 ** 64 - 1) for w in c.mask.tolist()]
        clear = [i for i, w in enumerate(words) if not (w >> hit) & 1]
        seen = [i for i, w in enumerate(words) if (w >> hit) & 1]
        assert clear and seen
        good = c.run()
        c.spoil(0, 37 + hit, value, which)
        got = c.run()
        c2 = good.double().cpu()[clear]
        # the spoiled strip's products run in fp32, so the bits may differ by a rounding
        out, *sizes = ref.attention(c.q, c.cache, c.table, c.ctx, c.start, c.mask, c.scale)
        bound = ref.attention_bound(fmt, 128, out, *sizes)[clear]
        assert ((got.double().cpu()[clear] - out[clear]).abs() <= bound).all()
        assert ((c2 - out[clear]).abs() <= bound).all()
        if which == "v" or value != value:                  # (an infinite key may score minus infinity: weight zero)
            assert not torch.isfinite(got[seen]).all(-1).any()


@pytest.mark.parametrize("fmt", FMTS)
def test_far_scores(fmt):
    """Scores of thousands, rising along the context: the running maximum moves all the time."""
    c = Case(fmt, 128, 2, 4, [700], [3], seed=11, spread=20.0, junk=False)
    c.check()


@pytest.mark.parametrize("fmt", FMTS)
def test_small_and_large_queries(fmt):
    """Rows from 2^-120 to 2^60 next to each other (their exponents are taken out before fp16)."""
    c = Case(fmt, 128, 1, 8, [90], [2], seed=12)
    e = torch.tensor([-120, -60, -20, -3, 0, 4, -126, -133], dtype=torch.float64)
    c.q[:] = (c.q.double() * (2.0 ** e).cuda()[None, :, None]).to(torch.bfloat16)
    c.check()
    c.q[:, 2] = 0
    c.check()


def test_strided_queries_streams_and_graphs():
    c = Case(bqg.Q8_0, 128, 2, 4, [200, 33], [3, 1], page=32, seed=13)
    wide = torch.full((c.n, c.H * 128 + 64), 9.0, dtype=torch.bfloat16, device="cuda")
    part = wide[:, :c.H * 128].unflatten(-1, (c.H, 128))
    part.copy_(c.q)
    want = c.run()
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
    for _ in range(2):
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_one_workspace_for_calls_of_different_shapes():
    big = Case(bqg.BF16, 256, 2, 4, [3000], [64], page=64, seed=1)
    small = [Case(f, D, 2, g, [5000], [t], page=64, seed=2) for f in FMTS for D, g, t in ((64, 1, 1), (128, 8, 9), (256, 2, 3))]
    ws = torch.zeros(max(c.ws.numel() for c in [big, *small]), dtype=torch.uint8, device="cuda")
    for c in [big, *small, big]:
        c.ws = ws
        c.check()


def test_bad_pages_and_lengths_are_reported():
    c = Case(bqg.Q8_0, 128, 2, 2, [100], [2], page=16, seed=5)
    keep = c.table.clone()
    for bad in (-1, c.cache.n_pages, 2 ** 31 - 1):
        c.table[0, 3] = bad                                 # tokens 48 .. 63 are not seen
        got = c.run()
        assert bqg.last_device_error() == bqg.DEVERR_PAGE
        c.table.copy_(keep)
        ctx = Case(bqg.Q8_0, 128, 2, 2, [84], [2], page=16, seed=5)      # the same without them
        ctx.q = c.q
        order = torch.tensor([i for i in range(7) if i != 3])
        ctx.table = keep[:, order.cuda()].contiguous()
        ctx.cache = c.cache
        ctx.check(got)
    c.check()
    c.ctx[0] = 10 ** 9                                      # beyond its pages: clamped to them
    c.run()
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH
    c.ctx[0] = -5
    got = c.run()
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH
    c.ctx[0] = 0
    c.check(got)
    for start in ([0, 99], [-3, 2], [2, 1]):
        c.start.copy_(torch.tensor(start, dtype=torch.int32))
        c.run()
        assert bqg.last_device_error() == bqg.DEVERR_LENGTH


def test_workspace_is_required():
    c = Case(bqg.BF16, 64, 1, 1, [5], [1])
    for ws in (None, c.ws[:-16]):
        with pytest.raises(bqg.BqgError) as e:
            bqg.tree_attention(c.q, c.cache, c.table, c.ctx, c.start, 1, ws=ws)
        assert e.value.status == 7
