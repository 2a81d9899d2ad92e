"""Attention behind shared prefixes directly behind the kernels that write what it reads, with dependent launches: its second pass begins
before its first one ends, and so without a wait of its own for them."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_cache_moves import i32, made, tensors
from test_gpu_tree_attention import FMTS

pytestmark = pytest.mark.gpu

PAGE, PREFIX, KV, GROUP, D = 16, 100, 2, 4, 128


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


class Chain:
    """Row 0 holds a prompt; the others become its branches; new tokens are written, and some of them moved."""

    def __init__(self, fmt, n, T):
        self.n, self.T, self.full = n, T, PREFIX // PAGE
        self.first = made(fmt, D, KV, PAGE, self.full + n + 20, 3)
        self.cache = made(fmt, D, KV, PAGE, self.full + n + 20, 3)
        dev = dict(device="cuda")
        self.table, self.ctx = torch.zeros((n, self.full + 2), dtype=torch.int32, **dev), torch.zeros(n, dtype=torch.int32, **dev)
        self.ctx2 = torch.zeros(n, dtype=torch.int32, **dev)
        self.parent, self.child, self.fresh = i32([0] * (n - 1)), i32(range(1, n)), i32([0] * (n - 1))
        self.start, self.prefix = i32(range(0, n * T + 1, T)), i32([PREFIX])
        self.q0 = torch.zeros((n * T, KV * GROUP, D), dtype=torch.bfloat16, **dev)
        self.q, self.k, self.v = (torch.zeros((n * T, h, D), **dev) for h in (KV * GROUP, KV, KV))
        self.slots, self.pos = torch.zeros(n * T, dtype=torch.int64, **dev), i32([PREFIX + t for _ in range(n) for t in range(T)])
        angle = torch.arange(256).double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.path, self.kept = torch.zeros((n, T), dtype=torch.int32, **dev), torch.zeros(n, dtype=torch.int32, **dev)
        self.q1 = torch.zeros_like(self.q0)
        self.outs = [torch.zeros_like(self.q0) for _ in range(3)]
        self.ws = bqg.shared_prefix_attention_workspace(self.cache, KV * GROUP, n, T, n * T)

    def inputs(self, seed):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        order = rng.permutation(self.full + self.n + 20)
        mine = order[self.full:self.full + self.n]                           # each row's page in use
        table = np.full((self.n, self.full + 2), -1)
        table[0, :self.full], table[0, self.full] = order[:self.full], mine[0]
        self.table.copy_(i32(table))
        self.ctx.copy_(i32([PREFIX] + [0] * (self.n - 1)))
        self.fresh.copy_(i32(mine[1:]))
        self.slots.copy_(torch.tensor([int(mine[b]) * PAGE + PREFIX % PAGE + t for b in range(self.n) for t in range(self.T)]))
        for x in (self.q0, self.q, self.k, self.v):
            x.copy_(torch.randn(x.shape, generator=g))
        kept = rng.integers(1, self.T + 1, self.n)
        self.kept.copy_(i32(kept))
        self.path.copy_(i32([[0] + sorted(rng.choice(np.arange(1, self.T), k - 1, replace=False).tolist()) + [-1] * (self.T - k)
                             for k in kept]).view(self.n, self.T))
        for old, t in zip(tensors(self.first), tensors(self.cache)):
            t.copy_(old)
        for t in (*self.outs, self.q1, self.ctx2):
            t.zero_()

    def attend(self, q, ctx, out):
        bqg.shared_prefix_attention(q, self.cache, self.table, ctx, self.start, self.T, self.prefix, out=out, ws=self.ws)

    def run(self, between=lambda: None):
        steps = [lambda: bqg.kv_fork(self.cache, self.table, self.ctx, self.parent, self.child, self.fresh),
                 lambda: self.attend(self.q0, self.ctx, self.outs[0]),
                 lambda: bqg.qk_norm_rope_kv_write(self.q, self.k, self.v, self.slots, self.cache, pos=self.pos, table=self.rope, out=self.q1),
                 lambda: self.attend(self.q1, self.ctx, self.outs[1]),
                 lambda: bqg.kv_compact(self.cache, self.table, self.ctx, self.path, self.kept, out=self.ctx2),
                 lambda: self.attend(self.q1, self.ctx2, self.outs[2])]
        for step in steps:
            step()
            between()

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (*self.outs, self.q1, self.ctx, self.ctx2, self.table)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,T", [(2, 1), (6, 3), (40, 4)])
def test_directly_behind_forks_writes_and_compactions(fmt, n, T):
    c = Chain(fmt, n, T)
    wants = []
    for seed in range(12):
        c.inputs(seed)
        c.run(torch.cuda.synchronize)
        wants.append(c.results())
        assert bqg.last_device_error() == 0
    assert all(t.float().abs().sum() > 0 for t in wants[0]) and not torch.equal(wants[0][1], wants[1][1])
    bqg.set_pdl(True)
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        for once in (g.replay, c.run):
            for seed, want in enumerate(wants):
                c.inputs(seed)
                once()
                for x, y in zip(c.results(), want):
                    assert torch.equal(x, y)
        assert bqg.last_device_error() == 0
    finally:
        bqg.set_pdl(False)
