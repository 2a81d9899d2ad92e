"""One layer's attention in speculative decoding, from the residual stream back to it.

    python examples/speculative_step.py

Per step: RMSNorm -> q8_1, the fused QKV GEMV, the queries' and keys' norm and rotation with the
write into the paged cache, attention, q8_1, the output projection.  Two sequences get a prompt
(causal), then each a tree of four drafted tokens, checked in one step; the accepted path's keys and
values then move to the places that follow the context.
"""
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import block_quantized_gemv_gb300 as bqg

EPS = 1e-5


class AttentionBlock:
    """Weights, cache and workspaces of one layer, laid out once."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, head_dim=128, fmt=bqg.Q8_0, n_pages=16, page=32, n_seq=2,
                 max_pages=6, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.K, self.H, self.KV, self.D, self.page = hidden, heads, kv_heads, head_dim, page
        self.Nq, self.Nkv = heads * head_dim, kv_heads * head_dim

        def weight(n, k):
            w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            return bqg.repack_weights(bqg.Q4_0, bqg.quantize_weights(bqg.Q4_0, w), n, k)

        self.Wq, self.Wk, self.Wv = weight(self.Nq, hidden), weight(self.Nkv, hidden), weight(self.Nkv, hidden)
        self.Wo = weight(hidden, self.Nq)
        self.gain = torch.ones(hidden, device="cuda")
        self.gain_q, self.gain_k = torch.ones(head_dim, device="cuda"), torch.ones(head_dim, device="cuda")
        at = torch.arange(max_pages * page, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, head_dim, 2, device="cuda") / head_dim)
        self.table = torch.cat([at.cos(), at.sin()], 1).contiguous()
        self.cache = bqg.kv_cache(fmt, n_pages, kv_heads, page, head_dim)
        # pages of the two sequences in any order
        order = torch.randperm(n_pages, generator=g, device="cuda")[:n_seq * max_pages]
        self.pages = order.view(n_seq, max_pages).to(torch.int32)
        self.ws = bqg.tree_attention_workspace(self.cache, heads, n_seq, 8)
        self.x = lambda m: torch.randn(m, hidden, generator=g, device="cuda").to(torch.bfloat16)

    def slots(self, seq, at):
        """Slots of places `at` of sequences `seq`."""
        return self.pages[seq, at // self.page].long() * self.page + at % self.page

    def step(self, x, seq, place, pos, ctx, q_start, max_q, mask=None):
        """x [M, hidden] (M <= 8): token i belongs to sequence seq[i], is stored at its place[i] and
        rotated to pos[i].  Returns the new residual, and the queries and attention it came from."""
        M = x.shape[0]
        xq = bqg.rmsnorm_quantize_q8_1(x, self.gain, EPS)
        q, k, v = bqg.gemv_q4_0_q8_1_qkv(self.Wq, self.Wk, self.Wv, xq, self.Nq, self.Nkv, self.K)
        q = bqg.qk_norm_rope_kv_write(q.view(M, self.H, self.D), k.view(M, self.KV, self.D), v.view(M, self.KV, self.D),
                                      self.slots(seq, place), self.cache, pos=pos, table=self.table, gamma_q=self.gain_q,
                                      gamma_k=self.gain_k, eps=EPS)
        a = bqg.tree_attention(q, self.cache, self.pages, ctx, q_start, max_q, mask=mask, ws=self.ws)
        y = bqg.gemv_q4_0_q8_1(self.Wo, bqg.quantize_q8_1(a.view(M, self.Nq)), self.K, self.Nq)
        return x + y, q, a

    def keep(self, seq, src, dst):
        """The tokens at places src of a sequence move to places dst."""
        k, v = bqg.kv_read(self.cache, self.slots(seq, src), dtype=torch.float32)
        bqg.kv_write(k, v, self.slots(seq, dst), self.cache)


def run(block, prompt=21, visit=None):
    """A prompt for both sequences, a drafted tree, the accepted path kept, one more token.  `visit` is
    called with every step's arguments and results."""
    def step(x, seq, place, pos, ctx, q_start, max_q, mask=None):
        t = lambda a, dt: torch.tensor(a, dtype=dt, device="cuda")
        args = (t(seq, torch.long), t(place, torch.long), t(pos, torch.int32), t(ctx, torch.int32),
                t(q_start, torch.int32), max_q, None if mask is None else t(mask, torch.long))
        out = block.step(x, *args)
        if visit:
            visit(args, out)
        return out[0]

    for at in range(0, prompt, 4):                                   # four tokens of each sequence at a time
        n = min(4, prompt - at)
        place = [at + i for _ in range(2) for i in range(n)]
        step(block.x(2 * n), [0] * n + [1] * n, place, place, [at, at], [0, n, 2 * n], n)
    # the tree: token 0, its two continuations 1 and 2, and 3 behind 2; each sees itself and its ancestors
    depth, sees = [0, 1, 1, 2], [0b0001, 0b0011, 0b0101, 0b1101]
    step(block.x(8), [0] * 4 + [1] * 4, [prompt + i for i in range(4)] * 2, [prompt + d for d in depth] * 2,
         [prompt, prompt], [0, 4, 8], 4, sees * 2)
    # say 0, 2, 3 are accepted: they follow the context now
    path = torch.tensor([prompt, prompt + 2, prompt + 3], device="cuda")
    for b in range(2):
        block.keep(torch.full((3,), b, device="cuda"), path, prompt + torch.arange(3, device="cuda"))
    return step(block.x(2), [0, 1], [prompt + 3] * 2, [prompt + 3] * 2, [prompt + 3] * 2, [0, 1, 2], 1)


if __name__ == "__main__":
    block = AttentionBlock()
    y = run(block)
    torch.cuda.synchronize()
    print("residual after the step:", tuple(y.shape), "device errors:", bqg.last_device_error())
