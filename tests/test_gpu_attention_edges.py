"""Attention where its operands leave the ordinary, against fp64, each sequence at once."""
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_tree_attention import Case

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
