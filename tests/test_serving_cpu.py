"""Host side of attention behind shared prefixes, verification, compaction and forks, without a GPU: what the C boundary and
the binding refuse, before anything is launched."""
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from test_kv_attention_cpu import BAD_CACHES, FAKE, L, cache, small_cache, stub  # noqa: F401


def share(L, **kw):
    a = dict(table=FAKE, pages=10, ctx=FAKE, start=FAKE, n_seq=2, n=5, max_q=3, n_q=32, prefix=FAKE, seqs=FAKE, n_prefix=2,
             most=5, mask=None, scale=0.1, out=FAKE, ws=FAKE, ws_bytes=1 << 30)
    q, qs = kw.pop("q", FAKE), kw.pop("qs", 4096)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_shared_prefix_attention(q, qs, cache(**c) if c is not None else None, *a.values(), None)


def verify(L, **kw):
    a = dict(target=FAKE, draft=FAKE, dt=bqg.F32, ts=1000, ds=1000, vocab=1000, tokens=FAKE, parent=FAKE, start=FAKE, n_seq=2,
             n=5, max_q=3, u=FAKE, count=FAKE, path=FAKE, token=FAKE)
    a.update(kw)
    return L.bqg_tree_verify(*a.values(), None)


def compact(L, **kw):
    a = dict(table=FAKE, pages=10, ctx=FAKE, path=FAKE + 128, n_path=FAKE + 256, n_seq=2, max_q=3, new=FAKE + 64)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_kv_compact(cache(**c) if c is not None else None, *a.values(), None)


def fork(L, **kw):
    a = dict(table=FAKE, pages=10, rows=4, ctx=FAKE, parent=FAKE, child=FAKE, fresh=FAKE, n=2)
    c = kw.pop("cache", {})
    a.update(kw)
    return L.bqg_kv_fork(cache(**c) if c is not None else None, *a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, status):
    for call in (share, compact, fork):
        assert call(L, cache=bad) == status
    assert L.bqg_shared_prefix_attention_workspace_size(cache(**bad), 32, 2, 3, 5, 1, 5) == 0


@pytest.mark.parametrize("call,kw,status", [
    (share, dict(cache=None), 1), (share, dict(q=None), 1), (share, dict(out=None), 1), (share, dict(table=None), 1),
    (share, dict(ctx=None), 1), (share, dict(start=None), 1), (share, dict(prefix=None), 1), (share, dict(seqs=None), 1),
    (share, dict(n_prefix=0), 1), (share, dict(n_prefix=-1), 1), (share, dict(most=-1), 1), (share, dict(n_seq=-1), 1),
    (share, dict(n=-1), 1), (share, dict(max_q=0), 1), (share, dict(pages=0), 1), (share, dict(n_q=33), 1),
    (share, dict(scale=0.0), 1), (share, dict(scale=float("nan")), 1), (share, dict(qs=4000), 1),
    (share, dict(most=(1 << 28) + 1), 2), (share, dict(max_q=65), 2), (share, dict(n=129), 2), (share, dict(n_q=8 * 65, qs=1 << 20), 2),
    (share, dict(pages=1 << 32), 2),
    (share, dict(q=FAKE + 2), 3), (share, dict(out=FAKE + 8), 3), (share, dict(table=FAKE + 2), 3), (share, dict(mask=FAKE + 4), 3),
    (share, dict(prefix=FAKE + 1), 3), (share, dict(seqs=FAKE + 2), 3), (share, dict(ws=FAKE + 4), 3),
    (verify, dict(target=None), 1), (verify, dict(tokens=None), 1), (verify, dict(start=None), 1), (verify, dict(u=None), 1),
    (verify, dict(count=None), 1), (verify, dict(path=None), 1), (verify, dict(token=None), 1), (verify, dict(dt=bqg.Q8_0), 1),
    (verify, dict(vocab=0), 1), (verify, dict(ts=999), 1), (verify, dict(ds=999), 1), (verify, dict(n_seq=-1), 1),
    (verify, dict(n=-1), 1), (verify, dict(max_q=0), 1),
    (verify, dict(max_q=65), 2), (verify, dict(n=129), 2), (verify, dict(vocab=(1 << 30) + 1, ts=1 << 31, ds=1 << 31), 2),
    (verify, dict(n_seq=1 << 28), 2), (verify, dict(ts=1 << 41), 2),
    (verify, dict(target=FAKE + 2), 3), (verify, dict(draft=FAKE + 1), 3), (verify, dict(dt=bqg.BF16, target=FAKE + 1), 3),
    (verify, dict(tokens=FAKE + 2), 3), (verify, dict(parent=FAKE + 2), 3), (verify, dict(u=FAKE + 1), 3), (verify, dict(path=FAKE + 2), 3),
    (compact, dict(cache=None), 1), (compact, dict(table=None), 1), (compact, dict(ctx=None), 1), (compact, dict(path=None), 1),
    (compact, dict(n_path=None), 1), (compact, dict(n_seq=-1), 1), (compact, dict(max_q=0), 1), (compact, dict(pages=0), 1),
    (compact, dict(new=FAKE), 1), (compact, dict(new=FAKE + 4), 1), (compact, dict(ctx=FAKE + 68), 1),
    (compact, dict(new=FAKE + 260), 1), (compact, dict(new=FAKE + 148), 1),
    (compact, dict(max_q=65), 2), (compact, dict(pages=1 << 32), 2),
    (compact, dict(table=FAKE + 2), 3), (compact, dict(path=FAKE + 1), 3), (compact, dict(new=FAKE + 66), 3),
    (fork, dict(cache=None), 1), (fork, dict(table=None), 1), (fork, dict(ctx=None), 1), (fork, dict(parent=None), 1),
    (fork, dict(child=None), 1), (fork, dict(fresh=None), 1), (fork, dict(n=-1), 1), (fork, dict(rows=-1), 1), (fork, dict(pages=0), 1),
    (fork, dict(pages=1 << 32), 2), (fork, dict(table=FAKE + 2), 3), (fork, dict(child=FAKE + 1), 3),
])
def test_bad_arguments_are_refused(L, call, kw, status):
    assert call(L, **kw) == status


def test_good_arguments_reach_the_device_check(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the fake pointers must not reach it")
    for call in (share, verify, compact, fork):
        assert call(L) in (4, 5)
    assert share(L, seqs=None, n_prefix=1) in (4, 5)
    assert share(L, n=0, n_seq=0, q=None, out=None, table=None, ctx=None, start=None, prefix=None) in (4, 5)
    assert verify(L, draft=None, ds=0, parent=None) in (4, 5)
    assert verify(L, dt=bqg.BF16, target=FAKE + 2, draft=FAKE + 6) in (4, 5)
    assert verify(L, n=0, target=None, tokens=None, u=None) in (4, 5)
    assert compact(L, new=None) in (4, 5) and compact(L, new=FAKE + 8) in (4, 5)
    assert fork(L, n=0, parent=None, child=None, fresh=None) in (4, 5)


# --- the binding ------------------------------------------------------------------
I32 = dict(dtype=torch.int32)


def test_shared_attention_arguments(stub):
    c = small_cache(bqg.Q4_0)
    q = torch.zeros(5, 6, 64, dtype=torch.bfloat16)
    good = dict(q=q, cache=c, block_table=torch.zeros(2, 4, **I32), ctx_len=torch.zeros(2, **I32), q_start=torch.zeros(3, **I32),
                max_q=4, prefix_len=torch.zeros(2, **I32), seq_start=torch.zeros(3, **I32), mask=torch.zeros(5, dtype=torch.int64))
    bqg.shared_prefix_attention(**good)
    a = stub[-1][1]
    assert a[4] == 4 and a[7:11] == (2, 5, 4, 6) and a[13:15] == (2, 5) and abs(a[16] - 0.125) < 1e-9
    bqg.shared_prefix_attention(**{**good, "prefix_len": torch.zeros(1, **I32), "seq_start": None, "max_shared": 3})
    assert stub[-1][1][12:15] == (None, 1, 3)
    n = len(stub)
    for key, bad in (("block_table", torch.zeros(4, **I32)), ("ctx_len", torch.zeros(3, **I32)), ("q_start", torch.zeros(2, **I32)),
                     ("seq_start", torch.zeros(2, **I32)), ("seq_start", None), ("mask", torch.zeros(4, dtype=torch.int64)),
                     ("q", torch.zeros(5, 6, 32, dtype=torch.bfloat16)), ("out", torch.zeros(5, 5, 64, dtype=torch.bfloat16)),
                     ("block_table", torch.zeros(4, 2, **I32).t())):
        with pytest.raises(ValueError):
            bqg.shared_prefix_attention(**{**good, key: bad})
    for key, bad in (("q", q.float()), ("prefix_len", torch.zeros(2)), ("seq_start", torch.zeros(3, dtype=torch.int64)),
                     ("mask", torch.zeros(5, **I32))):
        with pytest.raises(TypeError):
            bqg.shared_prefix_attention(**{**good, key: bad})
    assert len(stub) == n


def test_verification_arguments(stub, monkeypatch):
    monkeypatch.setattr(bqg, "_rows_checked", lambda t, name, shape, dtype: (16, bqg._row_stride(t, name, shape, dtype)))
    wide = torch.zeros(5, 300)
    good = dict(target=wide[:, :100], tokens=torch.zeros(5, **I32), q_start=torch.zeros(3, **I32), max_q=4, u=torch.zeros(5),
                parent=torch.zeros(5, **I32), draft=torch.zeros(5, 100))
    out = bqg.tree_verify(**good)
    assert [tuple(t.shape) for t in out] == [(2,), (2, 4), (2,)] and all(t.dtype == torch.int32 for t in out)
    a = stub[-1][1]
    assert a[2:6] == (bqg.F32, 300, 100, 100) and a[9:12] == (2, 5, 4)
    bqg.tree_verify(**{**good, "parent": None, "draft": None})
    assert stub[-1][1][1] is None and stub[-1][1][4] == 0 and stub[-1][1][7] is None
    n = len(stub)
    for key, bad in (("target", torch.zeros(500)), ("target", wide[:, :200:2]), ("draft", torch.zeros(5, 99)), ("tokens", torch.zeros(4, **I32)),
                     ("parent", torch.zeros(6, **I32)), ("u", torch.zeros(4)), ("q_start", torch.zeros(0, **I32)),
                     ("out", (torch.zeros(2, **I32), torch.zeros(2, 3, **I32), torch.zeros(2, **I32)))):
        with pytest.raises(ValueError):
            bqg.tree_verify(**{**good, key: bad})
    for key, bad in (("target", torch.zeros(5, 100, dtype=torch.float16)), ("draft", torch.zeros(5, 100, dtype=torch.bfloat16)),
                     ("tokens", torch.zeros(5, dtype=torch.int64)), ("u", torch.zeros(5, dtype=torch.float64)), ("q_start", torch.zeros(3))):
        with pytest.raises(TypeError):
            bqg.tree_verify(**{**good, key: bad})
    assert len(stub) == n


def test_compaction_and_fork_arguments(stub):
    c = small_cache(bqg.Q8_0)
    table, two = torch.zeros(2, 4, **I32), torch.zeros(2, **I32)
    good = dict(cache=c, block_table=table, ctx_len=two, path=torch.zeros(2, 5, **I32), n_path=torch.zeros(2, **I32))
    assert bqg.kv_compact(**good).shape == (2,)
    assert stub[-1][1][2] == 4 and stub[-1][1][6:8] == (2, 5)
    forks = dict(cache=c, block_table=table, ctx_len=two, parent=torch.zeros(3, **I32), child=torch.zeros(3, **I32), fresh=torch.zeros(3, **I32))
    bqg.kv_fork(**forks)
    assert stub[-1][1][2:4] == (4, 2) and stub[-1][1][8] == 3
    n = len(stub)
    for key, bad in (("block_table", two), ("ctx_len", torch.zeros(3, **I32)), ("path", torch.zeros(3, 5, **I32)), ("path", two),
                     ("n_path", torch.zeros(1, **I32)), ("out", torch.zeros(3, **I32)), ("path", torch.zeros(5, 2, **I32).t())):
        with pytest.raises(ValueError):
            bqg.kv_compact(**{**good, key: bad})
    for key, bad in (("block_table", table.long()), ("path", torch.zeros(2, 5)), ("n_path", two.long())):
        with pytest.raises(TypeError):
            bqg.kv_compact(**{**good, key: bad})
    for key, bad in (("block_table", two), ("ctx_len", torch.zeros(3, **I32)), ("child", two), ("fresh", two)):
        with pytest.raises(ValueError):
            bqg.kv_fork(**{**forks, key: bad})
    for key, bad in (("block_table", table.long()), ("parent", torch.zeros(3)), ("fresh", torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            bqg.kv_fork(**{**forks, key: bad})
    assert len(stub) == n
