"""Plain forms of the cache and attention entries, on the CPU: fp32 step by
step where include/bqgemv.h fixes the roundings (numpy, one IEEE operation
at a time), fp64 for attention."""
import numpy as np
import torch

import block_quantized_gemv_gb300 as bqg


def bf16_rn(x):
    """fp32 array -> bf16 values (nearest even), as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def norm_rope(x, norm, gamma, eps, pos, table, interleaved):
    """x fp32 [T, H, D] -> fp32, each rounding as the header states."""
    x = np.asarray(x, dtype=np.float32)
    T, H, D = x.shape
    y = x.copy()
    if norm:
        s = (x.astype(np.float64) ** 2).sum(-1, keepdims=True)
        r = (1.0 / np.sqrt(s / D + np.float64(np.float32(eps)))).astype(np.float32)
        y = (x * r).astype(np.float32)
        if gamma is not None:
            y = (y * gamma[None, None]).astype(np.float32)
    if table is None:
        return y
    R = table.shape[1]
    c, s = table[pos][:, None, :R // 2], table[pos][:, None, R // 2:]
    i = np.arange(R // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., ib] = (a * s).astype(np.float32) + (b * c).astype(np.float32)
    return y


def encode(ora, fmt, x):
    """fp32 rows [..., D] -> (codes, scales) as the cache holds them; the
    block encoders are the oracle's."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    if fmt == bqg.BF16:
        return bf16_rn(x), None
    import oracle
    D = x.shape[-1]
    rows = int(np.prod(x.shape[:-1]))
    size = 34 if fmt == bqg.Q8_0 else 18
    raw = np.frombuffer(np.ascontiguousarray(ora.quantize(oracle.Q8_0 if fmt == bqg.Q8_0 else oracle.Q4_0,
                                                           x.reshape(rows, D))).tobytes(), dtype=np.uint8)
    raw = raw.reshape(rows, D // 32, size)
    scales = raw[..., :2].copy().view(np.float16)[..., 0].reshape(*x.shape[:-1], D // 32)
    codes = raw[..., 2:].reshape(*x.shape[:-1], -1)
    return (codes.view(np.int8) if fmt == bqg.Q8_0 else codes).copy(), scales


def decode(fmt, codes, scales):
    """What the cache holds -> the exact values, fp64."""
    if fmt == bqg.BF16:
        return codes.astype(np.float64)
    d = np.repeat(scales.astype(np.float64), 32, axis=-1)
    if fmt == bqg.Q8_0:
        return codes.astype(np.float64) * d
    c = codes.reshape(*codes.shape[:-1], -1, 16)
    q = np.concatenate([c & 15, c >> 4], axis=-1).astype(np.float64) - 8
    return q.reshape(*codes.shape[:-1], -1) * d


def cache_values(cache):
    """(k, v) of a KVCache as fp64 arrays [n_pages, n_kv, page, D]."""
    out = []
    for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c = codes.float().cpu().numpy() if cache.fmt == bqg.BF16 else codes.cpu().numpy()
        out.append(decode(cache.fmt, c, None if scales is None else scales.cpu().numpy()))
    return out


def attention(q, cache, block_table, ctx_len, q_start, mask, scale):
    """fp64 attention and, for the tolerance, per output: sum_j p_j |v_j| and
    sum_j |v_j|, and per row the largest scale * sum_d |q_d k_jd|.  Each row
    sums over what it sees alone."""
    q = q.double().cpu()
    k, v = (torch.from_numpy(t) for t in cache_values(cache))
    n, H, D = q.shape
    P, KV = cache.page_size, cache.n_kv
    G = H // KV
    out, mag, every = (torch.zeros(n, H, D).double() for _ in range(3))
    reach = torch.zeros(n, H).double()
    table, ctx_len, q_start = block_table.cpu().long(), ctx_len.tolist(), q_start.tolist()
    words = None if mask is None else [int(w) & (2 ** 64 - 1) for w in mask.tolist()]
    for b in range(len(ctx_len)):
        T, ctx = q_start[b + 1] - q_start[b], ctx_len[b]
        at = torch.arange(ctx + T)
        page = table[b][at // P]
        kb, vb = k[page, :, at % P], v[page, :, at % P]                 # [L, KV, D]
        for i in range(T):
            see = [j for j in range(T) if (j <= i if words is None else (words[q_start[b] + i] >> j) & 1)]
            idx = torch.tensor(list(range(ctx)) + [ctx + j for j in see], dtype=torch.long)
            if len(idx) == 0:
                continue
            row = q_start[b] + i
            qr = q[row].view(KV, G, D)
            s = torch.einsum("hgd,lhd->hgl", qr, kb[idx]) * scale
            p = torch.softmax(s, -1)
            out[row] = torch.einsum("hgl,lhd->hgd", p, vb[idx]).reshape(H, D)
            mag[row] = torch.einsum("hgl,lhd->hgd", p, vb[idx].abs()).reshape(H, D)
            every[row] = vb[idx].abs().sum(0).repeat_interleave(G, 0)
            reach[row] = (torch.einsum("hgd,lhd->hgl", qr.abs(), kb[idx].abs()) * scale).amax(-1).reshape(H)
    return out, mag, every, reach


def attention_bound(fmt, dim, out, mag, every, reach):
    """How far a bf16 output may be from the exact one: half a step of bf16
    on the result (2^-8); the probabilities' rounding (bf16 2^-8, fp16
    2^-11) and, quantized, the values' (fp16 2^-11) on sum p |v|; the
    scores' fp32 accumulation, at most (dim + 8) roundings of 2^-24 (twice
    that for the tensor cores, which truncate) of the largest partial sum,
    moving each probability and their sum by that; the exponential
    and the fp32 sums: 2^-20."""
    u = 2.0 ** -8 if fmt == bqg.BF16 else 2.0 ** -11 + 2.0 ** -11
    floor = 0.0 if fmt == bqg.BF16 else 2.0 ** -33
    score = 2 * (dim + 8) * 2.0 ** -23 * reach
    return 2.0 ** -8 * out.abs() + (u + 2.0 ** -20 + score[..., None]) * mag * (1 + 2.0 ** -7) + floor * every + 1e-30
