"""Fork, attention behind the shared prompt, verification and compaction together, as the example runs them."""
import importlib.util
import sys
from pathlib import Path

import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from test_gpu_verify import verify

pytestmark = pytest.mark.gpu


def example():
    at = Path(__file__).resolve().parent.parent / "examples"
    sys.path.insert(0, str(at))
    try:
        spec = importlib.util.spec_from_file_location("branched_step", at / "branched_step.py")
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    finally:
        sys.path.remove(str(at))
    return mod


def held(block, b, places):
    """Codes and scales at places of sequence b, as bytes."""
    P = block.page
    at = [(int(block.pages[b, p // P]), p % P) for p in places]
    return [torch.stack([t.view(torch.int16 if t.element_size() == 2 else torch.int8)[page, :, off] for page, off in at])
            for t in (block.cache.k, block.cache.v, block.cache.k_scale, block.cache.v_scale) if t is not None]


@pytest.mark.parametrize("fmt", [bqg.BF16, bqg.Q8_0, bqg.Q4_0])
@pytest.mark.parametrize("prompt", [32, 40])                  # whole pages, and a part of one
def test_branches(fmt, prompt):
    mod = example()
    block = mod.Branches(fmt=fmt)
    T, rounds = mod.T, []

    def visit(tokens, ctx, prefix, out):
        if out is None:
            return
        (probs, u, kept, path, token), new, (q, a) = out
        want = verify(probs.cpu(), tokens.tolist(), [T, T], u.tolist(), mod.PARENT * 2, None, T)
        assert (kept.tolist(), path.tolist(), token.tolist()) == want
        assert new.tolist() == (ctx + kept).tolist()
        rounds.append((q, a, ctx.clone(), path.tolist(), kept.tolist()))

    # the drafts' places are written over by the compaction: each step is looked at as it is made
    real = bqg.kv_compact
    checked = []

    def watch(cache, pages, ctx, path, kept):
        before = [held(block, b, [int(ctx[b]) + i for i in path[b, :int(kept[b])].tolist()]) for b in range(2)]
        old = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
        new = real(cache, pages, ctx, path, kept)
        after = [held(block, b, range(int(ctx[b]), int(new[b]))) for b in range(2)]
        assert all(torch.equal(x, y) for p, r in zip(before, after) for x, y in zip(p, r))
        # the prompt stays as it was
        for b in range(2):
            for t, o in zip((t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None), old):
                for p in range(prompt):
                    page, off = int(pages[b, p // block.page]), p % block.page
                    assert torch.equal(t[page, :, off].view(torch.uint8), o[page, :, off].view(torch.uint8))
        checked.append(kept)
        return new

    mod.bqg.kv_compact = watch
    attention = []
    plain = bqg.shared_prefix_attention

    def attend(q, cache, pages, ctx, start, max_q, prefix, **kw):
        out = plain(q, cache, pages, ctx, start, max_q, prefix, **kw)
        want = ref.attention(q, cache, pages, ctx, start, kw["mask"], block.D ** -0.5)
        bound = ref.attention_bound(fmt, block.D, *want)
        if fmt != bqg.BF16:         # more than 16 rows behind the prompt: its keys are rounded to fp16, 2^-11 of each
            bound = bound + torch.expm1(2 * 2.0 ** -11 * want[3])[..., None] * want[2] * (1 + 2.0 ** -7)
        assert ((out.double().cpu() - want[0]).abs() <= bound).all()
        attention.append(out)
        return out

    mod.bqg.shared_prefix_attention = attend
    try:
        answers = mod.run(block, prompt=prompt, visit=visit)
    finally:
        mod.bqg.kv_compact, mod.bqg.shared_prefix_attention = real, plain
    assert len(attention) == len(checked) == len(rounds) == 3
    assert all(len(a) >= 3 for a in answers)
    # full pages are shared, the others are not
    full = prompt // block.page
    assert block.pages[0, :full].tolist() == block.pages[1, :full].tolist()
    assert not set(block.pages[0, full:].tolist()) & set(block.pages[1, full:].tolist())
    assert bqg.last_device_error() == 0
