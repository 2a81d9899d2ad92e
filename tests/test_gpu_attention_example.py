"""The example that runs norm, rotation, cache and attention together with the GEMVs around them."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref

pytestmark = pytest.mark.gpu


def example():
    path = Path(__file__).resolve().parent.parent / "examples" / "speculative_step.py"
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("fmt", [bqg.BF16, bqg.Q8_0, bqg.Q4_0])
def test_speculative_step(fmt):
    """Every step's attention against the fp64 form over what the cache then holds."""
    mod = example()
    block = mod.AttentionBlock(fmt=fmt)
    steps = []

    def visit(args, out):
        _, _, _, ctx, q_start, _, mask = args
        y, q, a = out
        want = ref.attention(q, block.cache, block.pages, ctx, q_start, mask, block.D ** -0.5)
        bound = ref.attention_bound(fmt, block.D, *want)
        assert ((a.double().cpu() - want[0]).abs() <= bound).all()
        assert torch.isfinite(y).all()
        steps.append(a.shape[0])

    y = mod.run(block, visit=visit)
    assert steps == [8, 8, 8, 8, 8, 2, 8, 2] and y.shape == (2, block.K)
    assert bqg.last_device_error() == 0


def test_the_kept_path_is_what_the_tree_held():
    """Moving tokens: a block's decoded values encode to themselves, but for the last bit of its scale."""
    mod = example()
    block = mod.AttentionBlock(fmt=bqg.Q8_0)
    held = []
    block_keep = block.keep

    def keep(seq, src, dst):
        before = bqg.kv_read(block.cache, block.slots(seq, src), dtype=torch.float32)
        block_keep(seq, src, dst)
        held.append((before, bqg.kv_read(block.cache, block.slots(seq, dst), dtype=torch.float32)))

    block.keep = keep
    mod.run(block)
    assert len(held) == 2
    for before, after in held:
        for x, y in zip(before, after):
            # the scale is fp16(amax / 127): off by at most 2^-11 of itself, codes then by at most half a step of it
            step = x.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True) / 127
            limit = (step * (0.5 + 127 * 2.0 ** -11)).expand(*step.shape[:-1], 32).flatten(-2)
            assert ((x - y).abs() <= limit * 1.001).all()


@pytest.mark.parametrize("fmt", [bqg.BF16, bqg.Q4_0])
@pytest.mark.parametrize("head_dim,kv_heads", [(128, 2), (256, 1), (64, 1)])
def test_dependent_launches_change_nothing(fmt, head_dim, kv_heads):
    """Programmatic dependent launch on: each kernel starts under the one before it and waits; the bits are the same."""
    mod = example()
    got = []
    for on in (False, True):
        block = mod.AttentionBlock(fmt=fmt, head_dim=head_dim, kv_heads=kv_heads, seed=3)
        was = bqg.set_pdl(on)
        try:
            got.append([mod.run(block).clone() for _ in range(3)])
            torch.cuda.synchronize()
        finally:
            bqg.set_pdl(was)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bqg.last_device_error() == 0
