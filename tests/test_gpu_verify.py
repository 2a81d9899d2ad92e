"""Verification of drafted tokens against the definition in exact arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


def verify(target, tokens, lens, u, parent, draft, max_q, number=Fraction):
    """The header's definition, sequence by sequence.  Fraction: exact; float: fp64."""
    V = target.shape[1]
    clean = lambda row: [number(min(x, 1.0)) if x > 0 else number(0) for x in row.tolist()]
    accepted, paths, nexts, start = [], [], [], 0
    for n in lens:
        path, nxt = [], -1
        if n:
            node, path = 0, [0]
            while True:
                p = clean(target[start + node])
                q = None if draft is None else clean(draft[start + node])
                r, Z, c, hit = p, number(1), number(0), None
                for i in range(node + 1, n):
                    if (i - 1 if parent is None else parent[start + i]) != node or not 0 <= tokens[start + i] < V:
                        continue
                    t = tokens[start + i]
                    if number(u[start + i]) * (1 if q is None else q[t]) * Z < r[t]:
                        hit = i
                        break
                    if q is None:
                        Z -= r[t]
                        r = list(r)
                        r[t] = number(0)
                    else:
                        c += Z
                        r = [max(a - c * b, number(0)) for a, b in zip(p, q)]
                        Z = sum(r)
                if hit is None:
                    break
                node = hit
                path.append(hit)
            if not sum(r) > 0:
                r = p
            total, run = sum(r), number(0)
            for x in range(V):
                run += r[x]
                if run > number(u[start]) * total:
                    nxt = x
                    break
        accepted.append(len(path))
        paths.append(path + [-1] * (max_q - len(path)))
        nexts.append(nxt)
        start += n
    return accepted, paths, nexts


class Case:
    def __init__(self, V, lens, dtype=torch.float32, drafted=True, chain=False, seed=0, sharp=2.0, near=0.5, max_q=None):
        rng = np.random.default_rng(seed)
        n = sum(lens)
        x = rng.normal(size=(n, V)) * sharp
        y = x + rng.normal(size=(n, V)) * near
        soft = lambda z: torch.softmax(torch.from_numpy(z), -1).to(dtype)
        self.target, self.draft, self.lens = soft(x), soft(y) if drafted else None, lens
        self.parent, self.tokens = [], []
        for T in lens:
            first = len(self.tokens)
            for i in range(T):
                up = i - 1 if chain else int(rng.random() ** 2 * i)
                self.parent.append(up if i else -1)
                if i == 0:
                    self.tokens.append(int(rng.integers(V)))
                elif drafted:
                    q = self.draft[first + up].double().numpy()
                    self.tokens.append(int(rng.choice(V, p=q / q.sum())))
                else:
                    nth = sum(self.parent[first + j] == up for j in range(1, i))
                    self.tokens.append(int(np.argsort(-y[first + up], kind="stable")[min(nth, V - 1)]))
        if chain:
            self.parent = None
        self.u = rng.random(n).astype(np.float32)
        self.u = np.minimum(self.u, np.float32(1 - 2.0 ** -24))
        self.max_q = max_q or max(max(lens), 1)

    def args(self):
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        start = np.concatenate([[0], np.cumsum(self.lens)])
        return dict(target=self.target.cuda(), tokens=i32(self.tokens), q_start=i32(start), max_q=self.max_q,
                    u=torch.from_numpy(np.asarray(self.u, dtype=np.float32)).cuda(),
                    parent=None if self.parent is None else i32(self.parent),
                    draft=None if self.draft is None else self.draft.cuda())

    def want(self, number=Fraction):
        return verify(self.target, self.tokens, self.lens, [float(x) for x in self.u], self.parent, self.draft, self.max_q, number)

    def check(self, got=None, number=Fraction, error=0):
        got = bqg.tree_verify(**self.args()) if got is None else got
        assert tuple(t.tolist() for t in got) == self.want(number)
        assert bqg.last_device_error() == error


@pytest.mark.parametrize("V", [1, 2, 31, 33, 300, 4099])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("chain", [False, True])
def test_chains_and_trees(V, dtype, drafted, chain):
    for seed in range(3):
        Case(V, [6, 1, 0, 13, 2, 0, 9], dtype, drafted, chain, seed=seed, sharp=1.0 + seed).check()


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("near", [0.05, 3.0])
def test_largest_trees(drafted, near):
    """64 tokens, drafts that are mostly accepted, and that are mostly rejected, many behind one token."""
    for seed in range(4):
        Case(70, [64, 64, 33], torch.float32, drafted, False, seed=seed, near=near).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("V", [16384, 32001, 131075])
def test_large_vocabularies(dtype, drafted, V):
    Case(V, [4, 7, 1], dtype, drafted, False, seed=V, sharp=3.0).check(number=float)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drafted", [False, True])
def test_many_large_vocabularies(dtype, drafted):
    """More sequences than have sixteen warps per CTA, more tokens than a warp's kept sums are single steps of."""
    Case(140001, [1, 2] * 18, dtype, drafted, False, seed=5, sharp=3.0).check(number=float)


@pytest.mark.parametrize("drafted", [False, True])
def test_the_largest_vocabularies(drafted):
    Case(600011, [3, 1], torch.bfloat16, drafted, False, seed=6, sharp=3.0).check(number=float)


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("u", [0.0, 1 - 2.0 ** -24])
def test_smallest_and_largest_numbers(drafted, u):
    c = Case(1000, [5, 1, 9], torch.float32, drafted, False, seed=3)
    c.u[:] = u
    c.check()
    c.u[:] = 1 - 2.0 ** -24                                   # rejected where they can be; the first token that is left
    c.u[[0, 5, 6]] = 0.0
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_draft_that_is_the_target_is_accepted(dtype):
    c = Case(500, [20], dtype, True, True, seed=1)
    c.draft = c.target.clone()
    c.check()
    assert bqg.tree_verify(**c.args())[0].item() == 20


def test_a_border_in_the_running_sum():
    """Probabilities and u that meet exactly: the sum has to exceed u times the whole."""
    for V in (4, 64, 4096):
        for k in range(0, V, max(1, V // 16)):
            c = Case(V, [1], torch.float32, False, True)
            c.target = torch.full((1, V), 1.0 / V)
            c.u[0] = k / V
            c.check()
            assert bqg.tree_verify(**c.args())[2].item() == k


def test_a_rejected_draft_is_not_taken_again():
    c = Case(8, [4], torch.float32, False, False, seed=2)
    c.parent, c.tokens = [-1, 0, 0, 0], [0, 5, 5, 2]          # twice the same chosen token
    c.target[0] = torch.tensor([0.1, 0.1, 0.0, 0.1, 0.1, 0.4, 0.1, 0.1])
    c.u[:] = [0.55, 0.9, 0.9, 0.0]
    c.check()


def test_nothing_left_and_nothing_there():
    c = Case(6, [2, 1, 1], torch.float32, False, True, seed=2)
    c.target[0] = torch.tensor([0.0, 0.0, 0.4, 0.0, 0.0, 0.0])   # one token, rejected: taken all the same
    c.tokens[1], c.u[1] = 2, 0.9
    c.target[2] = 0.0                                         # no probability at all
    c.target[3] = torch.tensor([float("nan"), -1.0, float("inf"), 0.25, -float("inf"), 0.25])
    c.check()
    assert bqg.tree_verify(**c.args())[2].tolist()[:2] == [2, -1]
    d = Case(6, [2], torch.float32, True, True, seed=2)
    d.target[0], d.draft[0] = torch.tensor([0.2, 0.0, 0.0, 0.0, 0.0, 0.0]), torch.full((6,), 0.3)
    d.tokens[1], d.u[1] = 0, 0.9
    d.check()


@pytest.mark.parametrize("drafted", [False, True])
def test_bad_drafts_and_offsets_are_reported(drafted):
    c = Case(50, [6, 5], torch.float32, drafted, False, seed=4, near=0.01)
    good = list(c.tokens), list(c.parent)
    for bad in (-1, 50, 2 ** 31 - 1):
        c.tokens[2] = bad
        c.check(error=bqg.DEVERR_DRAFT)
    c.tokens = list(good[0])
    for bad in (-1, 2, 5, 2 ** 31 - 1):                       # not before token 2
        c.parent[2] = bad
        got = bqg.tree_verify(**c.args())
        assert bqg.last_device_error() == bqg.DEVERR_DRAFT
        c.parent[2] = 77                                      # (whatever it is, nobody's child)
        assert tuple(t.tolist() for t in got) == c.want()
    c.parent = good[1]
    c.check()
    a = c.args()
    for start in ([0, 99, 11], [-3, 6, 11], [6, 2, 11], [1, 6, 11], [0, 6, 10]):
        a["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        bqg.tree_verify(**a)
        # (shifted tokens' parents need not stand before them: that is reported too)
        assert bqg.last_device_error() & ~bqg.DEVERR_DRAFT == bqg.DEVERR_LENGTH
    a = c.args()
    a["max_q"] = 3                                            # the rest of each sequence is left out
    got = bqg.tree_verify(**a)
    assert bqg.last_device_error() == bqg.DEVERR_LENGTH and got[1].shape == (2, 3) and int(got[0].max()) <= 3


def test_sampled_tokens_are_distributed_as_the_target():
    """30,000 sequences of one drafted tree: the first token given out, against the target, within five standard deviations."""
    N, V = 30000, 5
    rng = np.random.default_rng(0)
    p, q = np.array([0.1, 0.4, 0.05, 0.25, 0.2]), np.array([0.3, 0.1, 0.3, 0.2, 0.1])
    rows = np.stack([p, np.full(V, 0.2), np.full(V, 0.2)]).astype(np.float32)
    c = Case(V, [3], torch.float32, True, False)
    c.lens, c.max_q = [3] * N, 3
    c.target = torch.from_numpy(np.tile(rows, (N, 1)))
    c.draft = torch.from_numpy(np.tile(q.astype(np.float32), (3 * N, 1)))
    c.parent = [-1, 0, 0] * N
    c.tokens = np.stack([np.zeros(N), rng.choice(V, N, p=q), rng.choice(V, N, p=q)], 1).reshape(-1).astype(int).tolist()
    c.u = rng.random(3 * N).astype(np.float32)
    kept, path, nxt = (t.cpu().numpy() for t in bqg.tree_verify(**c.args()))
    tok = np.array(c.tokens).reshape(N, 3)
    given = np.where(kept == 1, nxt, tok[np.arange(N), np.maximum(path[:, 1], 0)])
    count = np.bincount(given, minlength=V)
    assert (np.abs(count - N * p) <= 5 * np.sqrt(N * p * (1 - p))).all(), count
    assert 0.2 < (kept > 1).mean() < 1


def test_strides_streams_and_graphs():
    c = Case(1001, [5, 8, 1], torch.float32, True, False, seed=6)
    a = c.args()
    want = bqg.tree_verify(**a)
    c.check(want)
    wide = torch.full((14, 2100), 0.5, device="cuda")
    wide[:, 3:1004], wide[:, 1050:2051] = a["target"], a["draft"]
    b = dict(a, target=wide[:, 3:1004], draft=wide[:, 1050:2051])
    for pdl in (False, True):
        bqg.set_pdl(pdl)
        try:
            assert all(torch.equal(x, y) for x, y in zip(bqg.tree_verify(**b), want))
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                got = bqg.tree_verify(**a)
            side.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            out = tuple(torch.zeros_like(t) for t in want)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                bqg.tree_verify(**a, out=out)
            for t in out:
                t.fill_(7)
            g.replay()
            assert all(torch.equal(x, y) for x, y in zip(out, want))
        finally:
            bqg.set_pdl(False)


def test_many_sequences():
    lens = np.random.default_rng(1).integers(0, 5, 700).tolist()
    Case(40, lens, torch.bfloat16, True, False, seed=8).check()
