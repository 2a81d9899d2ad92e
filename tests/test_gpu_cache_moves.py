"""The accepted path moved, and sequences branched, against the same on copies of the whole cache."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_tree_attention import FMTS, fill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def tensors(cache):
    return [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]


def raw(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def made(fmt, D, n_kv, page, n_pages, seed):
    c = bqg.kv_cache(fmt, n_pages, n_kv, page, D)
    fill(c, seed)
    return c


class Path:
    def __init__(self, fmt, D, n_kv, page, ctx, paths, max_q, seed=0):
        rng = np.random.default_rng(seed)
        per = (max(ctx) + 64 + page - 1) // page
        self.cache = made(fmt, D, n_kv, page, len(ctx) * per + 2, seed)
        self.table = rng.permutation(len(ctx) * per + 2)[:len(ctx) * per].reshape(len(ctx), per)
        self.ctx, self.paths, self.max_q = ctx, paths, max_q

    def want(self, skip=()):
        out = [raw(t).clone() for t in tensors(self.cache)]
        P = self.cache.page_size
        for b, path in enumerate(self.paths):
            for old, t in zip(tensors(self.cache), out):
                for k, a in enumerate(path):
                    x, y = self.ctx[b] + a, self.ctx[b] + k
                    if (b, k) not in skip:
                        t[self.table[b, y // P], :, y % P] = raw(old)[self.table[b, x // P], :, x % P]
        return out

    def args(self):
        rows = [list(p) + [-1] * (self.max_q - len(p)) for p in self.paths]
        return dict(block_table=i32(self.table), ctx_len=i32(self.ctx), path=i32(rows).view(len(self.ctx), self.max_q),
                    n_path=i32([len(p) for p in self.paths]))

    def check(self, error=0):
        want = self.want()
        ctx = bqg.kv_compact(self.cache, **self.args())
        assert ctx.tolist() == [c + len(p) for c, p in zip(self.ctx, self.paths)]
        for a, b in zip(tensors(self.cache), want):
            assert torch.equal(raw(a), b)
        assert bqg.last_device_error() == error


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,n_kv", [(16, 1), (32, 5), (128, 8)])
def test_paths(fmt, D, page, n_kv):
    """From nothing kept to all of 64; a place that is one token's source and another's goal; over the pages' ends."""
    paths = [[0, 2, 3], [], [0], list(range(64)), [0] + list(range(2, 64)), list(range(0, 64, 2)), [63], [5, 6, 40, 41, 63],
             list(range(32, 64)), [0, 1, 2, 9]]
    Path(fmt, D, n_kv, page, [0, 5, 15, 16, 17, 31, 100, 127, 128, 1], paths, 64, seed=page + D).check()


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences(fmt):
    rng = np.random.default_rng(2)
    paths = [sorted(rng.choice(9, rng.integers(0, 10), replace=False).tolist()) for _ in range(700)]
    Path(fmt, 128, 2, 16, rng.integers(0, 30, 700).tolist(), paths, 9, seed=3).check()


def test_bad_paths_are_cut_off():
    for path, good in (([0, 3, 3, 5], 2), ([0, 4, 2], 2), ([-1, 2], 0), ([0, 1, 2 ** 31 - 1], 2), ([2, 1000], 1)):
        c = Path(bqg.Q8_0, 128, 2, 16, [40, 7], [path, [0, 2]], 6, seed=1)
        a = c.args()
        c.paths[0] = path[:good]
        want = c.want()
        ctx = bqg.kv_compact(c.cache, **a)
        assert bqg.last_device_error() == bqg.DEVERR_LENGTH
        assert ctx.tolist() == [40 + good, 9]
        assert all(torch.equal(raw(x), y) for x, y in zip(tensors(c.cache), want))
    c = Path(bqg.Q8_0, 128, 2, 16, [40], [[0, 1, 3]], 3, seed=1)
    a = c.args()
    for n, kept in ((9, 3), (-2, 0)):                        # more or fewer than a path can hold
        a["n_path"] = i32([n])
        want = c.want() if kept else [raw(t).clone() for t in tensors(c.cache)]
        assert bqg.kv_compact(c.cache, **a).item() == 40 + kept
        assert bqg.last_device_error() == bqg.DEVERR_LENGTH
        assert all(torch.equal(raw(x), y) for x, y in zip(tensors(c.cache), want))


def test_bad_pages_are_left_out():
    for bad in (-1, 2 ** 31 - 1):
        c = Path(bqg.Q4_0, 128, 2, 16, [30], [[0, 3, 5, 20, 40]], 5, seed=1)      # from places 30, 33, 35, 50, 70
        good = int(c.table[0, 3])
        c.table[0, 3] = bad                                  # 48 .. 63
        a = c.args()
        c.table[0, 3] = good
        want = c.want(skip={(0, 3)})
        bqg.kv_compact(c.cache, **a)
        assert bqg.last_device_error() == bqg.DEVERR_PAGE
        assert all(torch.equal(raw(x), y) for x, y in zip(tensors(c.cache), want))


class Fork:
    def __init__(self, fmt, D, n_kv, page, ctx, pairs, seed=0, spare=2):
        """ctx: the parents' tokens; pairs: (parent, child) rows."""
        rng = np.random.default_rng(seed)
        rows = max([c for _, c in pairs] + [len(ctx) - 1]) + 1
        wide = max(ctx) // page + spare
        n_pages = len(ctx) * wide + len(pairs) + 3
        self.cache = made(fmt, D, n_kv, page, n_pages, seed)
        order = rng.permutation(n_pages)
        self.table = np.full((rows, wide), -7)
        self.table[:len(ctx)] = order[:len(ctx) * wide].reshape(len(ctx), wide)
        self.ctx = np.array(list(ctx) + [-9] * (rows - len(ctx)))
        self.pairs, self.fresh = pairs, order[len(ctx) * wide:len(ctx) * wide + len(pairs)].copy()

    def want(self, skip=(), keep=()):
        out, table, ctx, P = [raw(t).clone() for t in tensors(self.cache)], self.table.copy(), self.ctx.copy(), self.cache.page_size
        for i, (up, child) in enumerate(self.pairs):
            if i in skip:
                continue
            n = int(ctx[up])
            table[child, :n // P] = table[up, :n // P]
            if n // P < table.shape[1]:
                table[child, n // P] = self.fresh[i]
            ctx[child] = n
            if n % P and i not in keep:
                for t, old in zip(out, tensors(self.cache)):
                    t[self.fresh[i], :, :n % P] = raw(old)[self.table[up, n // P], :, :n % P]
        return out, table, ctx

    def check(self, skip=(), keep=(), error=0):
        want, table, ctx = self.want(skip, keep)
        t, c = i32(self.table), i32(self.ctx)
        bqg.kv_fork(self.cache, t, c, i32([p for p, _ in self.pairs]), i32([q for _, q in self.pairs]), i32(self.fresh))
        assert bqg.last_device_error() == error
        assert t.tolist() == table.tolist() and c.tolist() == ctx.tolist()
        assert all(torch.equal(raw(x), y) for x, y in zip(tensors(self.cache), want))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,n_kv", [(16, 1), (64, 5), (128, 8)])
def test_forks(fmt, D, page, n_kv):
    ctx = [0, 1, 15, 16, 17, 128, 200, 3, 127]
    pairs = [(6, 9), (6, 10), (6, 11), (0, 12), (1, 13), (2, 14), (3, 15), (4, 16), (5, 17), (7, 18), (8, 20), (8, 19)]
    Fork(fmt, D, n_kv, page, ctx, pairs, seed=page + D).check()


@pytest.mark.parametrize("fmt", FMTS)
def test_many_forks(fmt):
    rng = np.random.default_rng(5)
    Fork(fmt, 128, 3, 32, rng.integers(0, 700, 30).tolist(), [(int(rng.integers(30)), 30 + i) for i in range(800)], seed=4).check()


def test_a_full_row_has_no_next_page():
    f = Fork(bqg.BF16, 64, 2, 16, [64], [(0, 1)], spare=0)
    assert f.table.shape[1] == 4
    f.check()


def test_bad_forks_are_reported():
    new = lambda pairs: Fork(bqg.Q8_0, 128, 2, 16, [40, 20], pairs, seed=1)
    for bad in ((-1, 3), (9, 3), (2 ** 31 - 1, 3), (0, -1), (0, 99), (0, 0)):
        f = new([(1, 2), (0, 3)])
        f.pairs = [(1, 2), bad]
        f.check(skip={1}, error=bqg.DEVERR_ROW)
    for bad in (-1, 10 ** 6):
        f = new([(1, 2), (0, 3)])
        f.fresh[1] = bad                                     # entered, nothing copied
        f.check(keep={1}, error=bqg.DEVERR_PAGE)
    f = Fork(bqg.Q8_0, 128, 2, 16, [32], [(0, 1)], seed=1)
    f.fresh[0] = -1                                          # nothing to copy: no page needed yet
    f.check()
    f = new([(0, 2)])
    f.table[0, 2] = -4                                       # the parent's page in use
    f.check(keep={0}, error=bqg.DEVERR_PAGE)
    f = new([(0, 2)])
    f.ctx[0] = -5
    t, c = i32(f.table), i32(f.ctx)
    bqg.kv_fork(f.cache, t, c, i32([0]), i32([2]), i32(f.fresh))
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH and c.tolist()[2] == 0
    f.ctx[0] = 10 ** 9
    c = i32(f.ctx)
    bqg.kv_fork(f.cache, t, c, i32([0]), i32([2]), i32(f.fresh))
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH and c.tolist()[2] == f.table.shape[1] * 16


def test_streams_and_graphs():
    c = Path(bqg.Q8_0, 128, 2, 16, [40, 7], [[0, 2, 5], [1, 3]], 6, seed=1)
    first, want, a = [t.clone() for t in tensors(c.cache)], c.want(), c.args()
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bqg.kv_compact(c.cache, **a, out=out)
    f = Fork(bqg.Q4_0, 128, 2, 32, [70, 20], [(0, 2), (0, 3), (1, 4)], seed=1)
    fwant, table, ctx = f.want()
    t, n, ids = i32(f.table), i32(f.ctx), [i32([p for p, _ in f.pairs]), i32([q for _, q in f.pairs]), i32(f.fresh)]
    h = torch.cuda.CUDAGraph()
    with torch.cuda.graph(h):
        bqg.kv_fork(f.cache, t, n, *ids)
    for pdl in (False, True):
        bqg.set_pdl(pdl)
        try:
            for run in (g.replay, lambda: bqg.kv_compact(c.cache, **a, out=out)):
                for x, y in zip(tensors(c.cache), first):
                    x.copy_(y)
                run()
                assert out.tolist() == [43, 9]
                assert all(torch.equal(raw(x), y) for x, y in zip(tensors(c.cache), want))
            for run in (h.replay, lambda: bqg.kv_fork(f.cache, t, n, *ids)):
                t.copy_(i32(f.table)), n.copy_(i32(f.ctx))
                run()
                assert t.tolist() == table.tolist() and n.tolist() == ctx.tolist()
                assert all(torch.equal(raw(x), y) for x, y in zip(tensors(f.cache), fwant))
        finally:
            bqg.set_pdl(False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bqg.kv_compact(c.cache, **dict(a, n_path=i32([0, 0])))
    side.synchronize()
    assert got.tolist() == [40, 7]


def test_pages_beyond_32_bits_of_bytes():
    """A path and a fork at the end of a cache of more than 2^32 bytes a side."""
    n_kv, page, D = 2, 64, 128
    shift = 2 ** 32 // (n_kv * page * D * 2) + 1
    c = bqg.kv_cache(bqg.BF16, shift + 8, n_kv, page, D)
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in (c.k, c.v):
        t[shift:] = torch.randn(8, n_kv, page, D, generator=g, device="cuda").to(torch.bfloat16)
    k, v = c.k[shift:].clone(), c.v[shift:].clone()
    ctx, path = 60, [0, 3, 9]
    table = i32([[shift + 5, shift + 2]])
    assert bqg.kv_compact(c, table, i32([ctx]), i32([path]), i32([3])).item() == 63
    order = [5, 2]
    for old, t in ((k, c.k), (v, c.v)):
        want = old.clone()
        for i, a in enumerate(path):
            x, y = ctx + a, ctx + i
            want[order[y // page], :, y % page] = old[order[x // page], :, x % page]
        assert torch.equal(t[shift:], want) and not t[:8].any()
    k, v = c.k[shift:].clone(), c.v[shift:].clone()
    rows, n = i32([[shift + 5, shift + 2], [0, 0]]), i32([100, 0])
    bqg.kv_fork(c, rows, n, i32([0]), i32([1]), i32([shift + 7]))
    for old, t in ((k, c.k), (v, c.v)):
        want = old.clone()
        want[7, :, :36] = old[2, :, :36]
        assert torch.equal(t[shift:], want) and not t[:8].any()
    assert rows.tolist() == [[shift + 5, shift + 2], [shift + 5, shift + 7]] and n.tolist() == [100, 100]
    assert bqg.last_device_error() == 0
