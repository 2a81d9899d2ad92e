"""The cache's writer where a token is broken."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_gb300 as bqg
import kv_reference as ref
from block_quantized_gemv_gb300 import build as bqg_build
from test_gpu_kv_cache import FMTS, arrays, filled_cache, raw, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bqg_build.build()


@pytest.mark.parametrize("fmt", [bqg.Q8_0, bqg.Q4_0])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_block_with_a_nan_reads_as_nan(fmt, D, dtype):
    """Wherever in the block it is, and whatever else is there; the other blocks are what they are without it."""
    n_kv, page, T = 7, 32, 64
    rng = np.random.default_rng(D)
    clean = rng.standard_normal((T, n_kv, D), dtype=np.float32)
    clean[40, :, ::5], clean[41] = np.inf, 0.0
    clean[42, :, ::2], clean[42, :, 1::2] = -3.0, 3.0
    x = clean.copy()
    block = np.zeros((T, n_kv, D // 32), dtype=bool)
    for t in range(T):
        h, b = t % n_kv, t % (D // 32)
        x[t, h, 32 * b + t % 32] = np.nan
        block[t, h, b] = True
    x[7, 0, :32], block[7, 0, 0] = np.nan, True
    got = {}
    slots = torch.arange(T, device="cuda")
    for name, a in (("clean", clean), ("x", x)):
        cache = filled_cache(fmt, T // page, n_kv, page, D)
        key = torch.from_numpy(a).to(dtype).cuda()
        bqg.kv_write(key, key.flip(0).contiguous(), slots, cache)
        got[name] = arrays(cache), bqg.kv_read(cache, slots, dtype=torch.float32)
    for i, side in enumerate("kv"):
        hit = torch.from_numpy(block if side == "k" else block[::-1].copy())
        values = got["x"][1][i].cpu().unflatten(-1, (-1, 32))
        assert torch.isnan(values[hit]).all()
        place = lambda t: t.permute(0, 2, 1, 3).reshape(T, n_kv, D // 32, -1)              # [token, head, block, bytes]
        for n in (side, side + "_scale"):
            a, b = (place(got[v][0][n].view(torch.int16 if n.endswith("scale") else torch.uint8)) for v in ("clean", "x"))
            assert torch.equal(a[~hit], b[~hit])
    assert bqg.last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [8, 1000, -1])
def test_a_token_without_a_position_is_not_stored(ora, fmt, dtype, bad):
    """Neither its key nor its value: the place keeps the pair it had.  Its neighbours go in."""
    n_kv, page, D, T = 5, 16, 128, 4
    cache = filled_cache(fmt, 2, n_kv, page, D)
    before = arrays(cache)
    x = torch.from_numpy(np.random.default_rng(4).standard_normal((2, T, n_kv, D), dtype=np.float32)).to(dtype)
    pos = np.array([3, bad, 0, 7], dtype=np.int32)
    slots = [9, 17, 4, 30]
    table = rope_table(8, 64)
    q = bqg.qk_norm_rope_kv_write(x[0].cuda(), x[0].cuda(), x[1].cuda(), torch.tensor(slots, device="cuda"), cache,
                                  torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda())
    assert bqg.last_device_error() == bqg.DEVERR_POSITION
    assert not q[1].any() and q[[0, 2, 3]].any(-1).all()
    good = [0, 2, 3]
    after = arrays(cache)
    for name, t in (("k", ref.norm_rope(x[0, good].float().numpy(), 0, None, 0, pos[good], table, False)),
                    ("v", x[1, good].float().numpy())):
        codes, scales = ref.encode(ora, fmt, t)
        want = {name: torch.from_numpy(codes).to(before[name].dtype)}
        if scales is not None:
            want[name + "_scale"] = torch.from_numpy(scales)
        for n, w in want.items():
            full = before[n].clone()
            for i, t in enumerate(good):
                full[slots[t] // page, :, slots[t] % page] = w[i]
            assert np.array_equal(raw(after[n]), raw(full)), n


def test_errors_of_several_calls_come_together_and_once():
    """What different kernels report between two questions is in one word, which the question clears."""
    cache = bqg.kv_cache(bqg.Q8_0, 2, 1, 16, 64)
    x = torch.ones(1, 1, 64, device="cuda")
    at = lambda *v, dtype=torch.int32: torch.tensor(v, dtype=dtype, device="cuda")
    bqg.kv_read(cache, at(99, dtype=torch.int64))
    bqg.qk_norm_rope(x, x, at(5), torch.ones(2, 64, device="cuda"))
    for rows in (1, 40):
        q = torch.ones(rows, 1, 64, dtype=torch.bfloat16, device="cuda")
        ws = bqg.tree_attention_workspace(cache, 1, 1, rows)
        bqg.tree_attention(q, cache, at(-1, -1, -1).view(1, 3), at(0), at(0, rows), rows, ws=ws)
        seen = bqg.last_device_error()
        assert seen == (bqg.DEVERR_SLOT | bqg.DEVERR_POSITION | bqg.DEVERR_PAGE if rows == 1 else bqg.DEVERR_PAGE)
        assert bqg.last_device_error() == 0
