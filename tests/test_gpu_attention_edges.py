"""Attention where its operands leave the ordinary, against fp64, each sequence at once."""
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_tree_attention import FMTS, Case

pytestmark = pytest.mark.gpu

QUANT = [bqg.Q8_0, bqg.Q4_0]


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


def reference(c, gone=()):
    """fp64 attention of a Case without the places `gone` of its sequences, and the sizes of kv_reference.attention."""
    k, v = (torch.from_numpy(t).cuda() for t in ref.cache_values(c.cache))
    q, (n, H, D) = c.q.double(), c.q.shape
    KV, P = c.cache.n_kv, c.cache.page_size
    G = H // KV
    out, mag, every = (torch.zeros(n, H, D, dtype=torch.float64, device="cuda") for _ in range(3))
    reach = torch.zeros(n, H, dtype=torch.float64, device="cuda")
    start, ctx = c.start.tolist(), c.ctx.tolist()
    for b in range(len(ctx)):
        a, T = start[b], start[b + 1] - start[b]
        if T == 0:
            continue
        at = torch.arange(ctx[b] + T, device="cuda")
        sees = torch.ones(T, len(at), dtype=torch.bool, device="cuda")
        new = torch.arange(T, device="cuda")
        sees[:, ctx[b]:] = (new[None] <= new[:, None]) if c.mask is None else ((c.mask[a:a + T, None] >> new) & 1).bool()
        for place in gone:
            sees[:, place] = False
        page = c.table[b].long()[at // P]
        page = torch.where(sees.any(0), page, torch.zeros_like(page))
        kb, vb = k[page, :, at % P].transpose(0, 1), v[page, :, at % P].transpose(0, 1)            # [KV, L, D]
        dark = ~sees.any(0)
        kb[:, dark], vb[:, dark] = 0, 0
        rows = q[a:a + T].view(T, KV, G, D).permute(1, 0, 2, 3).reshape(KV, T * G, D)
        see = sees.repeat_interleave(G, 0)[None]
        s = (rows @ kb.transpose(1, 2) * c.scale).masked_fill(~see, -float("inf"))
        p = torch.softmax(s, -1).nan_to_num(0.0)                                                  # a row that sees nothing: zeros
        far = (rows.abs() @ kb.abs().transpose(1, 2) * c.scale).masked_fill(~see, 0.0).amax(-1)
        back = lambda t: t.view(KV, T, G, -1).permute(1, 0, 2, 3).reshape(T, H, -1)
        out[a:a + T], mag[a:a + T] = back(p @ vb), back(p @ vb.abs())
        every[a:a + T], reach[a:a + T] = back(see.double().expand_as(s) @ vb.abs()), back(far[..., None])[..., 0]
    return out, mag, every, reach


def bound(c, out, mag, every, reach):
    """kv_reference.attention_bound, and for more than 16 rows per KV head on quantized pages the keys' rounding to
    fp16: relative 2^-11 of each, so at most 2^-11 of the largest sum of |q k| on a score, which moves each
    probability by that factor and their sum by the same."""
    fmt, D = c.cache.fmt, c.cache.head_dim
    limit = ref.attention_bound(fmt, D, out, mag, every, reach)
    if fmt != bqg.BF16 and c.max_q * c.H // c.cache.n_kv > 16:
        limit = limit + torch.expm1(2 * 2.0 ** -11 * reach)[..., None] * mag * (1 + 2.0 ** -7)
    return limit


def within(c, got, gone=(), where=None):
    want = reference(c, gone)
    limit = bound(c, *want)
    ok = (got.double() - want[0]).abs() <= limit
    if where is not None:
        ok = ok | ~where
    assert ok.all(), ((got.double() - want[0]).abs() / limit)[~ok].max().item()


@pytest.mark.parametrize("fmt", QUANT)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group", [(5, 2), (30, 2), (64, 4)])
@pytest.mark.parametrize("which", ["v", "kv"])
def test_a_masked_value_beyond_fp16_reaches_nobody(fmt, D, T, group, which):
    """A drafted token whose codes times its finite scale pass 65504: a row that does not see it stays right, and so do
    the values of rows that see it wherever the token's own value is in range."""
    c = Case(fmt, D, 2, group, [37], [T], tree=True, seed=6)
    hit = 2
    c.spoil(0, 37 + hit, 1000.0 if fmt == bqg.Q8_0 else 20000.0, which)
    seen = ((c.mask >> hit) & 1).bool()
    assert seen.any() and not seen.all()
    place = 37 + hit
    value = torch.from_numpy(ref.cache_values(c.cache)[1]).cuda()[int(c.table[0, place // 16]), :, place % 16]   # [KV, D]
    assert (value.abs() > 65520).any() and (value.abs() < 65504).any()
    far = (value.abs() > 65504).repeat_interleave(group, 0)[None] & seen[:, None, None]
    if which == "kv":
        far = seen[:, None, None].expand_as(c.q)
    got = c.run()
    assert torch.isfinite(got[~seen]).all()
    within(c, got, where=~far)


@pytest.mark.parametrize("D,T,group", [(128, 2, 4), (128, 20, 4), (256, 20, 4)])
def test_queries_that_no_sequence_holds_are_reported(D, T, group):
    """q_start is to begin at 0 and end at the number of queries: others are in no sequence, and the call says so.
    The queries between are served."""
    c = Case(bqg.Q8_0, D, 2, group, [100, 40], [T, T], page=32, seed=14)
    keep = c.start.clone()
    for start in ([1, T, 2 * T], [0, T, 2 * T - 1], [2, T + 1, 2 * T - 1]):
        c.start.copy_(torch.tensor(start, dtype=torch.int32))
        got = c.run()
        assert bqg.last_device_error() == bqg.DEVERR_LENGTH
        within(c, got, where=((torch.arange(c.n, device="cuda") >= start[0])
                              & (torch.arange(c.n, device="cuda") < start[-1]))[:, None, None].expand_as(got))
    c.start.copy_(keep)
    within(c, c.run())
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group", [(1, 4), (3, 4), (9, 4), (30, 4), (64, 4)])
def test_the_maximum_rises_in_every_tile(fmt, D, T, group):
    """Keys that grow along the context, several tiles to a CTA: rows' maxima pass the former ones by far more than the
    slack, so what was summed up before is scaled down again and again."""
    c = Case(fmt, D, 8, group, [700] * 20, [T] * 20, page=64, tree=True, seed=7, junk=False)
    grow = torch.logspace(-1.5, 1.0, c.table.shape[1] * 64, dtype=torch.float64, device="cuda")
    t = c.cache.k if fmt == bqg.BF16 else c.cache.k_scale
    for b in range(20):
        pages = c.table[b].long()
        f = grow.view(-1, 1, 64, 1)
        t[pages] = (t[pages].double() * f).to(t.dtype)
    within(c, c.run())
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group", [(2, 4), (20, 4), (50, 4)])
@pytest.mark.parametrize("lost", [(1,), (2,), (0, 3, 6), (9,)])
def test_missing_pages_in_either_half_of_a_tile(fmt, D, T, group, lost):
    """Page numbers outside the cache, in the context and (page 9) among the new tokens: their tokens count for no row."""
    c = Case(fmt, D, 2, group, [300], [T], page=32, tree=True, seed=3, junk=False)
    for i, page in enumerate(lost):
        c.table[0, page] = (-1, c.cache.n_pages, 2 ** 31 - 1)[i]
    got = c.run()
    assert bqg.last_device_error() == bqg.DEVERR_PAGE
    within(c, got, gone=[32 * page + i for page in lost for i in range(32) if 32 * page + i < 300 + T])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,group", [(1, 1), (3, 4), (9, 4), (40, 4)])
def test_scales_of_either_sign(D, T, group):
    """q4_0: the scale has the sign of minus the block's largest value."""
    c = Case(bqg.Q4_0, D, 2, group, [333, 60], [T, 1], page=32, tree=True, seed=8)
    g = torch.Generator().manual_seed(9)
    for t in (c.cache.k_scale, c.cache.v_scale):
        t.mul_(torch.where(torch.rand(t.shape, generator=g) < 0.5, -1.0, 1.0).to(torch.float16).cuda())
    within(c, c.run())
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 3, 64])
def test_sixty_four_heads_per_kv_head(fmt, D, T):
    c = Case(fmt, D, 1, 64, [150, 7], [T, 1], page=16, tree=True, seed=T)
    within(c, c.run())
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,group", [(1, 4), (40, 4)])
def test_pages_beyond_32_bits_of_bytes(fmt, T, group):
    """The same pages at the end of a cache of more than 2^32 bytes a side: the same bits."""
    c = Case(fmt, 128, 2, group, [900, 130], [T, T], page=64, tree=True, seed=15)
    want = c.run()
    small = c.cache
    row = small.k[0].nbytes
    c.cache = bqg.kv_cache(fmt, 2 ** 32 // row + small.n_pages + 1, 2, 64, 128)
    at = c.cache.n_pages - small.n_pages
    for big, t in ((c.cache.k, small.k), (c.cache.v, small.v), (c.cache.k_scale, small.k_scale), (c.cache.v_scale, small.v_scale)):
        if t is not None:
            big[at:] = t
    c.table = c.table + at
    assert torch.equal(c.run().view(torch.int16), want.view(torch.int16))
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_workspace_for_more_new_tokens_serves_fewer(fmt, D):
    """A step checks trees of several sizes over one workspace, made for the largest."""
    cache = bqg.kv_cache(fmt, 1, 1, 16, D)
    for group in (1, 2, 3, 4, 5, 7, 8, 16, 64):
        sizes = [bqg.tree_attention_workspace(cache, group, 4, t).numel() for t in range(1, 65)]
        assert sizes == sorted(sizes), (group, sizes)
