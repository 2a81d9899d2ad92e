"""Two answers to one prompt, each by speculative decoding, over pages that they share.

    python examples/branched_step.py

The prompt goes into sequence 0 (causal), which is then forked: sequence 1 shares its full pages and has a copy of
the one in use.  Each round both get a drafted tree of four tokens; their attention reads the prompt once for both;
the target's probabilities accept a path and give the next token, whose number of the path's kept tokens move behind the
context, all without the host.
"""
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent))
from speculative_step import EPS, AttentionBlock, bqg

# token 0, its two drafts 1 and 2, and 3 behind 2; each sees itself and its ancestors
PARENT, DEPTH, SEES = [-1, 0, 0, 2], [0, 1, 1, 2], [0b0001, 0b0011, 0b0101, 0b1101]
T = len(PARENT)


class Branches(AttentionBlock):
    """The layer of speculative_step with an output projection to a vocabulary, and two sequences behind one prompt."""

    def __init__(self, vocab=512, fmt=bqg.Q8_0, seed=1, **kw):
        super().__init__(fmt=fmt, seed=seed, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        w = torch.randn(vocab, self.K, generator=g, device="cuda") * self.K ** -0.5
        self.vocab, self.Wout = vocab, bqg.repack_weights(bqg.Q4_0, bqg.quantize_weights(bqg.Q4_0, w), vocab, self.K)
        self.embed = torch.randn(vocab, self.K, generator=g, device="cuda").to(torch.bfloat16)
        self.u = lambda n: torch.rand(n, generator=g, device="cuda")
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        self.start, self.parent, self.depth = i32([0, T, 2 * T]), i32(PARENT * 2), i32(DEPTH * 2)
        self.sees = torch.tensor(SEES * 2, device="cuda")
        self.seq = torch.tensor([0] * T + [1] * T, device="cuda")
        self.at = torch.arange(T, device="cuda").repeat(2)
        self.shared_ws = bqg.shared_prefix_attention_workspace(self.cache, self.H, 2, T, 2 * T)

    def fork(self, ctx, fresh):
        """Sequence 1 becomes a branch of sequence 0."""
        one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
        bqg.kv_fork(self.cache, self.pages, ctx, one(0), one(1), one(fresh))

    def round(self, tokens, ctx, prefix):
        """tokens int32 [8]: both trees.  Returns the probabilities and what was accepted, the new context lengths, and the
        queries and attention on the way."""
        x = self.embed[tokens.long()]
        xq = bqg.rmsnorm_quantize_q8_1(x, self.gain, EPS)
        q, k, v = bqg.gemv_q4_0_q8_1_qkv(self.Wq, self.Wk, self.Wv, xq, self.Nq, self.Nkv, self.K)
        place = ctx[self.seq] + self.at
        q = bqg.qk_norm_rope_kv_write(q.view(2 * T, self.H, self.D), k.view(2 * T, self.KV, self.D), v.view(2 * T, self.KV, self.D),
                                      self.slots(self.seq, place), self.cache, pos=ctx[self.seq] + self.depth, table=self.table,
                                      gamma_q=self.gain_q, gamma_k=self.gain_k, eps=EPS)
        a = bqg.shared_prefix_attention(q, self.cache, self.pages, ctx, self.start, T, prefix, mask=self.sees, ws=self.shared_ws)
        y = x + bqg.gemv_q4_0_q8_1(self.Wo, bqg.quantize_q8_1(a.view(2 * T, self.Nq)), self.K, self.Nq)
        logits = bqg.gemv_q4_0_q8_1(self.Wout, bqg.rmsnorm_quantize_q8_1(y, self.gain, EPS), self.vocab, self.K)
        probs, u = torch.softmax(logits, -1), self.u(2 * T)
        kept, path, token = bqg.tree_verify(probs, tokens, self.start, T, u, parent=self.parent)
        return (probs, u, kept, path, token), bqg.kv_compact(self.cache, self.pages, ctx, path, kept), (q, a)


def run(block, prompt=40, rounds=3, visit=None):
    """Returns both answers' tokens.  `visit` is called with every round's arguments and results, before and after."""
    for at in range(0, prompt, 4):                                   # the prompt, four tokens at a time
        place = torch.arange(at, at + 4, device="cuda")
        block.step(block.x(4), torch.zeros(4, dtype=torch.long, device="cuda"), place, place.int(),
                   *(torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([at, 0], [0, 4, 4])), 4)
    ctx = torch.tensor([prompt, 0], dtype=torch.int32, device="cuda")
    block.fork(ctx, int(block.pages[1, prompt // block.page]))
    prefix = torch.tensor([prompt], dtype=torch.int32, device="cuda")
    tokens = torch.zeros(2 * T, dtype=torch.int32, device="cuda")
    answers = [[], []]
    for _ in range(rounds):
        if visit:
            visit(tokens, ctx, prefix, None)
        got, new, qa = block.round(tokens, ctx, prefix)
        if visit:
            visit(tokens, ctx, prefix, (got, new, qa))
        probs, _, kept, path, token = got
        for b in range(2):
            answers[b] += [int(tokens[b * T + i]) for i in path[b, 1:int(kept[b])]] + [int(token[b])]
        # the next trees: the new token, and the likeliest ones of the last accepted token's row as its drafts
        best = probs[torch.stack([path[b, int(kept[b]) - 1] + b * T for b in range(2)]).long()].topk(T - 1).indices.int()
        tokens, ctx = torch.cat([token[:, None], best], 1).reshape(-1).contiguous(), new
    return answers


if __name__ == "__main__":
    block = Branches()
    answers = run(block)
    torch.cuda.synchronize()
    print("answers:", answers, "device errors:", bqg.last_device_error())
