"""The cache's handle: what it was made with is what its calls use."""
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
from test_kv_attention_cpu import small_cache, stub  # noqa: F401


def test_its_tensors_and_sizes_cannot_be_replaced(stub):
    """The addresses are taken once: a tensor put in its place would not be the one that calls write to."""
    for fmt in (bqg.BF16, bqg.Q8_0, bqg.Q4_0):
        c = small_cache(fmt)
        kept = {n: getattr(c, n) for n in ("fmt", "n_pages", "n_kv", "page_size", "head_dim", "k", "v", "k_scale", "v_scale")}
        for name, value in kept.items():
            with pytest.raises(AttributeError):
                setattr(c, name, value.clone() if isinstance(value, torch.Tensor) else 1)
            assert getattr(c, name) is value
        c.k.fill_(1)                                        # their contents can
