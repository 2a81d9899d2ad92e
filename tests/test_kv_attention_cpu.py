"""Host side of the cache and attention entries, without a GPU: what the C
boundary and the binding refuse, before anything is launched."""
import ctypes

import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build

FAKE = 0x10000      # never dereferenced: every call below fails validation first, or finds no device


@pytest.fixture(scope="module")
def L():
    bqg_build.build()
    return bqg.load()


def cache(**kw):
    f = dict(fmt=bqg.Q8_0, page_size=64, n_kv=8, head_dim=128, n_pages=100, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE)
    f.update(kw)
    s = bqg._KVCacheStruct(**f)
    cache.keep = s
    return ctypes.addressof(s)


BAD_CACHES = [(dict(fmt=3), 1), (dict(fmt=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
              (dict(v_scale=None), 1), (dict(n_kv=0), 1), (dict(n_pages=0), 1), (dict(n_pages=-1), 1),
              (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
              (dict(page_size=8192), 2), (dict(page_size=-64), 2), (dict(n_pages=2 ** 50), 2), (dict(n_kv=2000), 2),
              (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3), (dict(k_scale=FAKE + 4), 3)]


def norm_rope(L, **kw):
    a = dict(q=FAKE, k=FAKE, dt=bqg.F32, qs=4096, ks=1024, T=3, n_q=32, n_kv=8, D=128, norm=1, gq=FAKE, gk=None,
             eps=1e-5, pos=FAKE, table=FAKE, n_pos=10, rot=128, inter=0, qo=FAKE, ko=FAKE)
    a.update(kw)
    return L.bqg_qk_norm_rope(*a.values(), None)


def norm_write(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dt=bqg.F32, qs=4096, ks=1024, vs=1024, T=3, n_q=32, norm=1, gq=FAKE, gk=None,
             eps=1e-5, pos=FAKE, table=FAKE, n_pos=10, rot=128, inter=0, qo=FAKE, slots=FAKE)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_qk_norm_rope_kv_write(*a.values(), cache(**c) if c is not None else None, None)


def write(L, **kw):
    a = dict(k=FAKE, v=FAKE, dt=bqg.BF16, ks=1024, vs=1024, T=3, slots=FAKE)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_kv_write(*a.values(), cache(**c) if c is not None else None, None)


def read(L, **kw):
    a = dict(slots=FAKE, T=3, dt=bqg.BF16, ko=FAKE, vo=FAKE)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_kv_read(cache(**c) if c is not None else None, *a.values(), None)


def attend(L, **kw):
    a = dict(table=FAKE, pages=10, ctx=FAKE, start=FAKE, n_seq=2, n=5, max_q=3, n_q=32, mask=None, scale=0.1, out=FAKE,
             ws=FAKE, ws_bytes=1 << 30)
    q, qs = kw.pop("q", FAKE), kw.pop("qs", 4096)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_tree_attention(q, qs, cache(**c) if c is not None else None, *a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, status):
    for call in (norm_write, write, read, attend):
        assert call(L, cache=bad) == status
    assert L.bqg_tree_attention_workspace_size(cache(**bad), 32, 2, 3) == 0


@pytest.mark.parametrize("call,kw,status", [
    (norm_rope, dict(dt=bqg.Q8_0), 1), (norm_rope, dict(T=-1), 1), (norm_rope, dict(q=None), 1),
    (norm_rope, dict(qo=None), 1), (norm_rope, dict(k=None), 1), (norm_rope, dict(ko=None), 1),
    (norm_rope, dict(n_q=-1), 1), (norm_rope, dict(norm=2), 1), (norm_rope, dict(eps=-1.0), 1),
    (norm_rope, dict(eps=float("nan")), 1), (norm_rope, dict(eps=float("inf")), 1), (norm_rope, dict(inter=5), 1),
    (norm_rope, dict(table=None), 1), (norm_rope, dict(pos=None), 1), (norm_rope, dict(n_pos=0), 1),
    (norm_rope, dict(qs=4095), 1), (norm_rope, dict(ks=1000), 1),
    (norm_rope, dict(D=80), 2), (norm_rope, dict(rot=24), 2), (norm_rope, dict(rot=144), 2), (norm_rope, dict(rot=-16), 2),
    (norm_rope, dict(n_q=1025, qs=1 << 20), 2), (norm_rope, dict(T=1 << 31), 2),
    (norm_rope, dict(q=FAKE + 8), 3), (norm_rope, dict(qs=4098), 3), (norm_rope, dict(dt=bqg.BF16, ks=1028), 3),
    (norm_rope, dict(qo=FAKE + 2), 3), (norm_rope, dict(table=FAKE + 4), 3), (norm_rope, dict(pos=FAKE + 2), 3),
    (norm_rope, dict(gq=FAKE + 4), 3),
    (norm_write, dict(cache=None), 1), (norm_write, dict(v=None), 1), (norm_write, dict(slots=None), 1),
    (norm_write, dict(vs=1020), 1), (norm_write, dict(slots=FAKE + 4), 3), (norm_write, dict(v=FAKE + 8), 3),
    (norm_write, dict(n_q=32, qo=None), 1),
    (write, dict(cache=None), 1), (write, dict(dt=7), 1), (write, dict(T=-2), 1), (write, dict(k=FAKE + 4), 3),
    (read, dict(cache=None), 1), (read, dict(dt=bqg.Q8_1), 1), (read, dict(T=-2), 1), (read, dict(ko=None), 1),
    (read, dict(slots=None), 1), (read, dict(vo=FAKE + 8), 3), (read, dict(slots=FAKE + 4), 3),
    (attend, dict(cache=None), 1), (attend, dict(q=None), 1), (attend, dict(out=None), 1), (attend, dict(table=None), 1),
    (attend, dict(ctx=None), 1), (attend, dict(start=None), 1), (attend, dict(n_seq=-1), 1), (attend, dict(n=-1), 1),
    (attend, dict(max_q=0), 1), (attend, dict(pages=0), 1), (attend, dict(n_q=0), 1), (attend, dict(n_q=33), 1),
    (attend, dict(scale=0.0), 1), (attend, dict(scale=-1.0), 1), (attend, dict(scale=float("nan")), 1),
    (attend, dict(scale=float("inf")), 1), (attend, dict(qs=4000), 1),
    (attend, dict(max_q=65), 2), (attend, dict(n_q=8 * 65, qs=1 << 20), 2), (attend, dict(n=129), 2),
    (attend, dict(pages=1 << 32), 2),
    (attend, dict(q=FAKE + 2), 3), (attend, dict(qs=4100), 3), (attend, dict(out=FAKE + 8), 3),
    (attend, dict(table=FAKE + 2), 3), (attend, dict(mask=FAKE + 4), 3), (attend, dict(ws=FAKE + 4), 3),
])
def test_bad_arguments_are_refused(L, call, kw, status):
    assert call(L, **kw) == status


def test_good_arguments_reach_the_device_check(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the fake pointers must not reach it")
    for call in (norm_rope, norm_write, write, read, attend):
        assert call(L) in (4, 5)
    assert write(L, T=0, k=None, v=None, slots=None) in (4, 5)
    assert norm_rope(L, T=0, q=None, k=None, qo=None, ko=None, pos=None) in (4, 5)
    assert norm_rope(L, rot=0, pos=None, table=None, n_pos=0) in (4, 5)
    assert norm_rope(L, n_kv=0, k=None, ko=None, ks=0) in (4, 5)
    assert read(L, cache=dict(fmt=bqg.BF16, k_scale=None, v_scale=None)) in (4, 5)
    assert L.bqg_tree_attention_workspace_size(cache(), 32, 2, 3) == 0


# --- the binding ------------------------------------------------------------------
@pytest.fixture
def stub(monkeypatch):
    """The binding over CPU tensors and a library that records its calls."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    def dev(t, name, dtype=None, numel=None):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        bqg._check_tensor(t, name, dtype, numel)
        return 16

    monkeypatch.setattr(bqg, "load", lambda path=None: Lib())
    monkeypatch.setattr(bqg, "_dev", dev)
    monkeypatch.setattr(bqg, "_tokens_checked", lambda t, name, shape, dtype: (16, bqg._token_stride(t, name, shape, dtype)))
    monkeypatch.setattr(bqg, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(bqg, "check_device", lambda *a: None)
    monkeypatch.setattr(bqg, "_current_device", lambda: 0)
    return calls


def small_cache(fmt):
    return bqg.kv_cache(fmt, 5, 2, 16, 64, device="cpu")


def test_the_cache_checks_its_tensors(stub):
    for fmt in (bqg.BF16, bqg.Q8_0, bqg.Q4_0):
        c = small_cache(fmt)
        assert (c.n_pages, c.n_kv, c.page_size, c.head_dim) == (5, 2, 16, 64)
        t = [c.k, c.v, c.k_scale, c.v_scale]
        with pytest.raises(ValueError):
            bqg.KVCache(fmt, t[0][0], t[1][0], *t[2:])
        with pytest.raises(ValueError):
            bqg.KVCache(fmt, t[0], t[1][1:], *t[2:])
        with pytest.raises(TypeError):
            bqg.KVCache(fmt, t[0].to(torch.float64), t[1], *t[2:])
        with pytest.raises(ValueError):
            bqg.KVCache(fmt, t[0].transpose(1, 2), t[1].transpose(1, 2), *t[2:])
    c = small_cache(bqg.Q8_0)
    for bad in ((None, c.v_scale), (c.k_scale[1:], c.v_scale), (c.k_scale.float(), c.v_scale)):
        with pytest.raises((ValueError, TypeError)):
            bqg.KVCache(bqg.Q8_0, c.k, c.v, *bad)
    b = small_cache(bqg.BF16)
    with pytest.raises(ValueError):
        bqg.KVCache(bqg.BF16, b.k, b.v, c.k_scale, c.v_scale)
    for f in (bqg.Q8_1, 9):
        with pytest.raises(ValueError):
            bqg.kv_cache(f, 1, 1, 16, 64, device="cpu")
        with pytest.raises(ValueError):
            bqg.KVCache(f, b.k, b.v)


def test_token_strides_are_passed_and_other_layouts_refused(stub):
    c = small_cache(bqg.Q8_0)
    rows = torch.zeros(4, (6 + 2 + 2) * 64 + 16)
    q, k, v = (rows[:, a * 64:(a + h) * 64].unflatten(-1, (h, 64)) for a, h in ((0, 6), (6, 2), (8, 2)))
    slots = torch.zeros(4, dtype=torch.int64)
    bqg.qk_norm_rope_kv_write(q, k, v, slots, c)
    name, a = stub[-1]
    assert name == "bqg_qk_norm_rope_kv_write" and a[4:7] == (656, 656, 656) and a[7:9] == (4, 6)
    bqg.kv_write(k, v, slots, c)
    assert stub[-1][1][3:5] == (656, 656)
    n = len(stub)
    for bad in (lambda: bqg.kv_write(k.transpose(0, 1), v, slots, c),
                lambda: bqg.kv_write(k[..., ::2], v, slots, c),
                lambda: bqg.kv_write(k, v[:3], slots, c),
                lambda: bqg.kv_write(k[:, :1], v, slots, c),
                lambda: bqg.kv_write(k, v, slots[:3], c),
                lambda: bqg.kv_write(k[0], v[0], slots, c),
                lambda: bqg.kv_write(torch.zeros(4, 2, 128)[..., :64], v, slots, c)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bqg.kv_write(k.half(), v, slots, c), lambda: bqg.kv_write(k, v.bfloat16(), slots, c),
                lambda: bqg.kv_write(k, v, slots.int(), c), lambda: bqg.kv_read(c, slots, dtype=torch.float16),
                lambda: bqg.qk_norm_rope(q.half(), k)):
        with pytest.raises(TypeError):
            bad()
    assert len(stub) == n


def test_norm_and_rotation_arguments(stub):
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    g, pos, table = torch.ones(64), torch.zeros(3, dtype=torch.int32), torch.zeros(9, 32)
    bqg.qk_norm_rope(q, k, pos, table, gamma_q=g, eps=1e-5, interleaved=True)
    a = stub[-1][1]
    assert a[9] == 1 and a[15:18] == (9, 32, 1)
    bqg.qk_norm_rope(q, k)
    assert stub[-1][1][9] == 0 and stub[-1][1][16] == 0
    n = len(stub)
    for bad in (dict(gamma_q=g), dict(pos=pos), dict(pos=pos[:2], table=table), dict(pos=pos, table=table[0]),
                dict(gamma_k=g[:32], eps=1e-5), dict(out=(torch.zeros(3, 4, 32, dtype=torch.bfloat16),) * 2)):
        with pytest.raises(ValueError):
            bqg.qk_norm_rope(q, k, **bad)
    for bad in (dict(pos=pos.long(), table=table), dict(pos=pos, table=table.double()), dict(pos=None, table=table),
                dict(gamma_q=g.half(), eps=1e-5)):
        with pytest.raises(TypeError):
            bqg.qk_norm_rope(q, k, **bad)
    assert len(stub) == n


def test_attention_arguments(stub):
    c = small_cache(bqg.Q4_0)
    i32 = dict(dtype=torch.int32)
    q = torch.zeros(5, 6, 64, dtype=torch.bfloat16)
    good = dict(q=q, cache=c, block_table=torch.zeros(2, 4, **i32), ctx_len=torch.zeros(2, **i32),
                q_start=torch.zeros(3, **i32), max_q=4, mask=torch.zeros(5, dtype=torch.int64))
    bqg.tree_attention(**good)
    a = stub[-1][1]
    assert a[4] == 4 and a[7:11] == (2, 5, 4, 6) and abs(a[12] - 0.125) < 1e-9
    n = len(stub)
    for key, bad in (("block_table", torch.zeros(4, **i32)), ("ctx_len", torch.zeros(3, **i32)),
                     ("q_start", torch.zeros(2, **i32)), ("mask", torch.zeros(4, dtype=torch.int64)),
                     ("q", torch.zeros(5, 6, 32, dtype=torch.bfloat16)), ("out", torch.zeros(5, 5, 64, dtype=torch.bfloat16)),
                     ("block_table", torch.zeros(4, 2, **i32).t())):
        with pytest.raises(ValueError):
            bqg.tree_attention(**{**good, key: bad})
    for key, bad in (("q", q.float()), ("block_table", torch.zeros(2, 4, dtype=torch.int64)), ("mask", torch.zeros(5, **i32)),
                     ("ctx_len", torch.zeros(2)), ("out", torch.zeros(5, 6, 64))):
        with pytest.raises(TypeError):
            bqg.tree_attention(**{**good, key: bad})
    assert len(stub) == n
