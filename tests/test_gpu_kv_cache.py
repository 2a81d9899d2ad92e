"""Per-head norm and rotation, and the paged cache's writer and reader, bit
for bit against the plain forms: every rounding is fixed by
include/bqgemv.h (r itself may differ in its last bit for about one row in
2^20; the seeds here hold none)."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from block_quantized_gemv_gb300 import build as bqg_build

pytestmark = pytest.mark.gpu

FMTS = [bqg.BF16, bqg.Q8_0, bqg.Q4_0]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


def rope_table(n_pos, rot):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rows(seed, T, n_q, n_kv, D, dtype, pad=0):
    """q, k, v as parts of one row per token (pad values between tokens), on the GPU, and as fp32 arrays."""
    g = np.random.default_rng(seed)
    w = (n_q + 2 * n_kv) * D + pad
    x = torch.from_numpy(g.standard_normal((T, w), dtype=np.float32)).to(dtype)
    parts = x.cuda()
    cut = lambda t, a, h: t[:, a * D:(a + h) * D].unflatten(-1, (h, D))
    dev = [cut(parts, 0, n_q), cut(parts, n_q, n_kv), cut(parts, n_q + n_kv, n_kv)]
    host = [cut(x.float(), 0, n_q).numpy(), cut(x.float(), n_q, n_kv).numpy(), cut(x.float(), n_q + n_kv, n_kv).numpy()]
    return dev, host


def filled_cache(fmt, n_pages, n_kv, page, D, seed=0):
    """A cache whose bytes are all 0x5a, to see what a call wrote."""
    c = bqg.kv_cache(fmt, n_pages, n_kv, page, D)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(0x5a)
    return c


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def expect_cache(cache, before, slots, k, v, ora):
    """The cache's arrays as they should be after k, v went to `slots`."""
    P = cache.page_size
    want = {n: t.clone() for n, t in before.items()}
    for name, x in (("k", k), ("v", v)):
        codes, scales = ref.encode(ora, cache.fmt, x)
        codes = torch.from_numpy(codes)
        if cache.fmt == bqg.BF16:
            codes = codes.to(torch.bfloat16)
        for t, slot in enumerate(slots):
            if slot < 0:
                continue
            want[name][slot // P, :, slot % P] = codes[t]
            if scales is not None:
                want[name + "_scale"][slot // P, :, slot % P] = torch.from_numpy(scales[t])
    return want


def arrays(cache):
    return {n: getattr(cache, n).cpu() for n in ("k", "v", "k_scale", "v_scale") if getattr(cache, n) is not None}


def check_cache(cache, want):
    for n, t in arrays(cache).items():
        assert np.array_equal(raw(t), raw(want[n])), n


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 96), (128, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [0, 1, 2])
def test_qk_norm_rope(D, rot, dtype, interleaved, norm):
    T, n_q, n_kv, n_pos = 9, 5, 3, 700
    (q, k, _), (qh, kh, _) = rows(D + rot + norm, T, n_q, n_kv, D, dtype, pad=8)
    g = np.random.default_rng(3)
    pos = g.integers(0, n_pos, T).astype(np.int32)
    table = rope_table(n_pos, rot) if rot else None
    gq, gk = ((1 + 0.2 * g.standard_normal(D)).astype(np.float32) for _ in range(2))
    kw = dict(gamma_q=torch.from_numpy(gq).cuda(), gamma_k=torch.from_numpy(gk).cuda()) if norm == 2 else {}
    got = bqg.qk_norm_rope(q, k, torch.from_numpy(pos).cuda() if rot else None,
                           torch.from_numpy(table).cuda() if rot else None, eps=EPS if norm else None,
                           interleaved=interleaved, **kw)
    for y, x, gain in zip(got, (qh, kh), (gq, gk)):
        want = ref.bf16_rn(ref.norm_rope(x, norm, gain if norm == 2 else None, EPS, pos, table, interleaved))
        assert np.array_equal(y.float().cpu().numpy(), want)
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n_q,n_kv,page", [(1, 4, 1, 16), (7, 7, 7, 32), (301, 6, 2, 64)])
def test_norm_rope_into_the_cache(ora, fmt, D, dtype, T, n_q, n_kv, page):
    n_pages, n_pos = (T + page - 1) // page + 2, 5000
    (q, k, v), (qh, kh, vh) = rows(T + D, T, n_q, n_kv, D, dtype)
    g = np.random.default_rng(5)
    pos = g.integers(0, n_pos, T).astype(np.int32)
    slots = g.permutation(n_pages * page)[:T].astype(np.int64)
    if T > 3:
        slots[[1, T - 1]] = -1
    table = rope_table(n_pos, D // 2)
    gk = (1 + 0.2 * g.standard_normal(D)).astype(np.float32)
    cache = filled_cache(fmt, n_pages, n_kv, page, D)
    before = arrays(cache)
    y = bqg.qk_norm_rope_kv_write(q, k, v, torch.from_numpy(slots).cuda(), cache, torch.from_numpy(pos).cuda(),
                                  torch.from_numpy(table).cuda(), gamma_k=torch.from_numpy(gk).cuda(), eps=EPS)
    assert np.array_equal(y.float().cpu().numpy(), ref.bf16_rn(ref.norm_rope(qh, 1, None, EPS, pos, table, False)))
    check_cache(cache, expect_cache(cache, before, slots, ref.norm_rope(kh, 1, gk, EPS, pos, table, False), vh, ora))
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_then_read(ora, fmt, D, dtype):
    T, n_kv, page, n_pages = 77, 3, 16, 9
    (_, k, v), (_, kh, vh) = rows(D, T, 1, n_kv, D, dtype)
    # blocks of zeros, tiny, huge and equal values, and ties of the largest magnitude
    kh[0, 0], kh[1, 0], kh[2, 0], kh[3, 0] = 0.0, 1e-30, 2.0 ** 17, 1.0
    kh[4, 0, ::2], kh[4, 0, 1::2] = -2.0, 2.0
    kh[5, 0, :32], kh[6, 0, 32:64] = 2.0 ** -25, -3.0 * 2.0 ** -24
    k = torch.from_numpy(kh).to(dtype).cuda()
    kh = k.float().cpu().numpy()
    slots = np.random.default_rng(1).permutation(n_pages * page)[:T].astype(np.int64)
    slots[10] = -7
    cache = filled_cache(fmt, n_pages, n_kv, page, D)
    before = arrays(cache)
    dslots = torch.from_numpy(slots).cuda()
    bqg.kv_write(k, v, dslots, cache)
    want = expect_cache(cache, before, slots, kh, vh, ora)
    check_cache(cache, want)
    exact = ref.cache_values(cache)
    stored = (slots >= 0)[:, None, None]
    for dt in (torch.float32, torch.bfloat16):
        for got, x in zip(bqg.kv_read(cache, dslots, dtype=dt), exact):
            w = np.where(stored, x[slots.clip(0) // page, :, slots.clip(0) % page], 0.0).astype(np.float32)
            if dt == torch.bfloat16:
                w = ref.bf16_rn(w)
            assert np.array_equal(got.float().cpu().numpy(), w)
    assert bqg.last_device_error() == 0


def test_no_tokens_and_one_side_only():
    cache = filled_cache(bqg.Q8_0, 2, 2, 16, 64)
    before = arrays(cache)
    e = torch.empty((0, 2, 64), device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    bqg.kv_write(e, e, none, cache)
    assert [t.shape for t in bqg.kv_read(cache, none)] == [(0, 2, 64)] * 2
    assert bqg.qk_norm_rope_kv_write(e, e, e, none, cache).shape == (0, 2, 64)
    check_cache(cache, before)
    x = torch.randn(3, 4, 64, device="cuda")
    q, k = bqg.qk_norm_rope(x, x[:, :0])                     # queries alone, nothing to do but the rounding
    assert torch.equal(q, x.to(torch.bfloat16)) and k.shape == (3, 0, 64)


def test_rows_beyond_the_pair_arithmetic():
    """Rows whose squares leave fp32's range, and rows of zeros."""
    D = 128
    x = np.random.default_rng(2).standard_normal((6, 1, D)).astype(np.float32)
    x[0] *= np.float32(2.0 ** 90)
    x[1] *= np.float32(2.0 ** -90)
    x[2] = 0
    x[3, 0, 1:] = 0
    x[4, 0, ::2] *= np.float32(2.0 ** 70)
    d = torch.from_numpy(x).cuda()
    for eps in (1e-5, 0.0):
        keep = [0, 1, 3, 4, 5] if eps == 0.0 else list(range(6))      # 1 / sqrt(0) for the row of zeros
        q, _ = bqg.qk_norm_rope(d, d, eps=eps)
        want = ref.bf16_rn(ref.norm_rope(x[keep], 1, None, eps, None, None, False))
        assert np.array_equal(q.float().cpu().numpy()[keep], want)


def test_out_of_range_slots_and_positions_are_reported():
    n_kv, page, D = 2, 16, 128
    cache = filled_cache(bqg.Q4_0, 3, n_kv, page, D)
    before = arrays(cache)
    x = torch.randn(2, n_kv, D, device="cuda")
    bad = torch.tensor([3 * page, 2 ** 45], dtype=torch.int64, device="cuda")
    bqg.kv_write(x, x, bad, cache)
    assert bqg.last_device_error() == bqg.DEVERR_SLOT and bqg.last_device_error() == 0
    check_cache(cache, before)
    k, v = bqg.kv_read(cache, bad)
    assert not k.any() and not v.any() and bqg.last_device_error() == bqg.DEVERR_SLOT
    table = torch.from_numpy(rope_table(8, 128)).cuda()
    ok = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    for p in ([8, 3], [-1, 3]):
        pos = torch.tensor(p, dtype=torch.int32, device="cuda")
        q = bqg.qk_norm_rope_kv_write(x, x, x, ok, cache, pos, table)
        assert not q[0].any() and q[1].any() and bqg.last_device_error() == bqg.DEVERR_POSITION
    # the token without a position left its key's place alone; its value went in
    assert np.array_equal(raw(cache.k[0, :, 1]), raw(before["k"][0, :, 1]))
    assert not np.array_equal(raw(cache.k[0, :, 2]), raw(before["k"][0, :, 2]))


def test_offsets_beyond_32_bits(ora):
    """A cache of more than 2^32 bytes: its last page."""
    n_kv, page, D = 8, 4096, 256
    n_pages = 2 ** 32 // (n_kv * page * D) + 3
    cache = bqg.kv_cache(bqg.Q8_0, n_pages, n_kv, page, D)
    (_, k, v), (_, kh, vh) = rows(1, 2, 1, n_kv, D, torch.float32)
    slots = torch.tensor([n_pages * page - 1, (n_pages - 1) * page], dtype=torch.int64, device="cuda")
    bqg.kv_write(k, v, slots, cache)
    for got, x in zip(bqg.kv_read(cache, slots, dtype=torch.float32), (kh, vh)):
        codes, scales = ref.encode(ora, bqg.Q8_0, x)
        assert np.array_equal(got.cpu().numpy(), ref.decode(bqg.Q8_0, codes, scales).astype(np.float32))
    assert not cache.k[:-1].view(-1)[:2 ** 31].any()


def test_on_another_stream_and_in_a_graph(ora):
    n_kv, page, D, T = 2, 16, 64, 5
    (q, k, v), (qh, kh, vh) = rows(8, T, 4, n_kv, D, torch.float32)
    slots = torch.arange(T, device="cuda")
    cache = filled_cache(bqg.Q8_0, 2, n_kv, page, D)
    before = arrays(cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bqg.kv_write(k, v, slots, cache)
    side.synchronize()
    check_cache(cache, expect_cache(cache, before, slots.tolist(), kh, vh, ora))
    out = torch.empty((T, 4, D), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bqg.qk_norm_rope_kv_write(q, k, v, slots, cache, eps=EPS, out=out)
    for t in (cache.k, cache.v):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.float().cpu().numpy(), ref.bf16_rn(ref.norm_rope(qh, 1, None, EPS, None, None, False)))
    want = expect_cache(cache, {n: torch.zeros_like(t) if n in "kv" else t for n, t in before.items()}, slots.tolist(),
                        ref.norm_rope(kh, 1, None, EPS, None, None, False), vh, ora)
    for n in ("k", "v"):
        assert np.array_equal(raw(getattr(cache, n).cpu()), raw(want[n]))
