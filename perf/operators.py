"""The attention side of a decode step over a block-quantized KV cache: cases, inputs and plain forms.

Three operators:

  rope   Per-head RMSNorm of queries and keys with the rotary position rotation, the keys and values going
         straight into a paged cache (bf16, q8_0 or q4_0).  Returns the queries and what the cache then holds.
  cache  New keys and values quantized into the cache, and a range of the cache read back.
  attn   Attention of each sequence's newest tokens (one token, a causal run, or a tree of drafted tokens under
         an ancestor mask) over its pages of the cache.

The cache is n_pages pages of `page` tokens for each KV head.  bf16: values.  q8_0: int8 codes and one fp16 scale
per 32 values, value q d, d = fp16(amax / 127).  q4_0: two codes per byte (element j low, j + 16 high, within 32),
value (q - 8) d, d = fp16(m / -8) for the first value m of largest magnitude.  Codes divide by the stored scale in
fp32 and round half away from zero.
"""
import math
import random

import torch

own = False

BF16, Q8_0, Q4_0 = "bf16", "q8_0", "q4_0"
EPS = 2.0 ** -20      # about 1e-6, and the same number in 32 bits
FRESH = 1.5     # spread of the attention's queries: scores of a few units, some keys stand out


# --- cases ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # the newest token of one chat of an 8B-style model (32 query heads on 8 KV heads): latency counts
        dict(name="rope 1 token q8_0", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, fmt=Q8_0, page=64,
             x="f32", norm=True, interleaved=False, start=4095, one_prompt=False, pad=0),
        # a 512-token prompt chunk of a 7B-style model (32 heads, each with keys of its own), adjacent-pair rotation
        dict(name="rope 512 tokens q4_0", op="rope", tokens=512, heads=32, kv_heads=32, dim=128, rot=128, fmt=Q4_0,
             page=32, x="f32", norm=False, interleaved=True, start=0, one_prompt=True, pad=0),
        # a ragged batch of prompt chunks at far positions, 64 query heads, half of each head rotated
        dict(name="rope 7001 tokens bf16", op="rope", tokens=7001, heads=64, kv_heads=8, dim=128, rot=64, fmt=BF16,
             page=16, x="bf16", norm=True, interleaved=False, start=120000, one_prompt=True, pad=3),
        # 33 new tokens, then one sequence of 4099 read back (to move or save it), small heads and pages
        dict(name="cache 33 into 4099 q8_0", op="cache", tokens=33, read=4099, kv_heads=8, dim=64, fmt=Q8_0, page=16,
             x="bf16"),
        # a prompt of 8192 tokens written and read back
        dict(name="cache 8192 q4_0", op="cache", tokens=8192, read=8192, kv_heads=8, dim=128, fmt=Q4_0, page=64,
             x="f32"),
        # one chat, one token, a short context: latency counts
        dict(name="attn 1x777 q8_0", op="attn", fmt=Q8_0, batch=1, ctx=777, tree=1, ragged=False, heads=32, kv_heads=8,
             dim=128, page=64, causal=True),
        # a serving batch of ragged chats, one token each
        dict(name="attn 32x8191 bf16", op="attn", fmt=BF16, batch=32, ctx=8191, tree=1, ragged=True, heads=32,
             kv_heads=8, dim=128, page=64, causal=True),
        # eight chats of a 7B-style model without shared heads
        dict(name="attn 8x4096 mha q4_0", op="attn", fmt=Q4_0, batch=8, ctx=4096, tree=1, ragged=False, heads=32,
             kv_heads=32, dim=128, page=32, causal=True),
        # one very long document, one token: the work has to be split along the context
        dict(name="attn 1x131071 q8_0", op="attn", fmt=Q8_0, batch=1, ctx=131071, tree=1, ragged=False, heads=32,
             kv_heads=8, dim=128, page=128, causal=True),
        # speculative decoding, small trees of drafted tokens
        dict(name="attn tree 8x5000 q8_0", op="attn", fmt=Q8_0, batch=8, ctx=5000, tree=13, ragged=True, heads=32,
             kv_heads=8, dim=128, page=64, causal=False),
        # the same with an odd number of query heads on each KV head and small pages
        dict(name="attn tree 16x2999 q4_0", op="attn", fmt=Q4_0, batch=16, ctx=2999, tree=32, ragged=True, heads=28,
             kv_heads=4, dim=128, page=16, causal=False),
        # wide trees over long contexts of a 70B-style model: bound by the products
        dict(name="attn tree 4x16384 bf16", op="attn", fmt=BF16, batch=4, ctx=16384, tree=64, ragged=False, heads=64,
             kv_heads=8, dim=128, page=64, causal=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng, most):
    kv = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    return kv * rng.choice([g for g in (1, 2, 3, 4, 4, 5, 7, 8, 16) if kv * g <= most]), kv


def draw(rng):
    op = rng.choice(["rope", "cache", "attn", "attn"])
    fmt = rng.choice([BF16, Q8_0, Q4_0])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    x = rng.choice(["f32", "bf16"])
    if op == "rope":
        heads, kv = _heads(rng, 64)
        most = max(1, min(8192, 70_000_000 // ((heads + 2 * kv) * dim)))
        tokens = _log(rng, 1, most)
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv, dim=dim,
                    rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128, 256) if r <= dim]), fmt=fmt, page=page, x=x,
                    norm=rng.random() < 0.6, interleaved=rng.random() < 0.4, start=_log(rng, 1, 130000),
                    one_prompt=rng.random() < 0.5, pad=rng.choice([0, 0, min(tokens - 1, 5)]))
    if op == "cache":
        kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
        read = _log(rng, 1, max(1, min(32768, 8_400_000 // (kv * dim))))
        return dict(op=op, tokens=_log(rng, 1, read), read=read, kv_heads=kv, dim=dim, fmt=fmt, page=page, x=x)
    heads, kv = _heads(rng, 64)
    causal = rng.random() < 0.4
    tree = rng.choice([1, 1, _log(rng, 1, 64)]) if causal else _log(rng, 2, 64)
    batch = _log(rng, 1, 64)
    # at most about the bytes and the products of the largest listed cases
    room = min(260_000_000 // (batch * kv * dim * 2), 34_000_000_000 // (batch * heads * tree * dim), 131071)
    return dict(op=op, fmt=fmt, batch=batch, ctx=_log(rng, 1, max(1, room - tree)), tree=tree,
                ragged=rng.random() < 0.6, heads=heads, kv_heads=kv, dim=dim, page=page, causal=causal)


# --- inputs --------------------------------------------------------------------------------------------------------
def _away(x):
    """Rounded to whole numbers, halves away from zero."""
    a = x.abs()
    t = a.trunc()
    return torch.sign(x) * (t + (a - t >= 0.5).to(x.dtype))


def _encode(x, fmt):
    """fp32 [..., dim] -> what the cache holds: (codes, scales), or (values, None)."""
    if fmt == BF16:
        return x.to(torch.bfloat16), None
    b = x.unflatten(-1, (-1, 32))
    if fmt == Q8_0:
        top = b.abs().amax(-1, keepdim=True)
        d = torch.div(top, torch.full_like(top, 127.0)).half()
        s = d.float().expand_as(b)
        q = torch.where(s == 0, torch.zeros_like(b), _away(torch.div(b, torch.where(s == 0, torch.ones_like(s), s))))
        return q.clamp(-127, 127).to(torch.int8).flatten(-2), d.squeeze(-1)
    a = b.abs()
    at = torch.arange(32, device=x.device).expand_as(b)
    first = torch.where(a == a.amax(-1, keepdim=True), at, torch.full_like(at, 32)).amin(-1, keepdim=True)
    m = b.gather(-1, first)
    d = torch.div(m, torch.full_like(m, -8.0)).half()
    s = d.float().expand_as(b)
    q = torch.where(s == 0, torch.zeros_like(b), _away(torch.div(b, torch.where(s == 0, torch.ones_like(s), s))))
    q = (q + 8).clamp(0, 15).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d.squeeze(-1)


def _decode(codes, scales, fmt):
    """What _encode gives -> fp32 values."""
    if fmt == BF16:
        return codes.float()
    if fmt == Q8_0:
        return (codes.float().unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)
    c = codes.unflatten(-1, (-1, 16))
    q = torch.cat([c & 15, c >> 4], -1).float() - 8.0
    return (q * scales.float().unsqueeze(-1)).flatten(-2)


def _normal(gen, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _empty_cache(gen, n_pages, kv, page, dim, fmt):
    """A cache as an allocator hands it out: whatever bytes were there."""
    def junk(last, dtype, size):
        n = n_pages * kv * page * last
        raw = torch.randint(0, 256, (n * size,), generator=gen, device="cuda", dtype=torch.uint8)
        return raw.view(dtype).view(n_pages, kv, page, last)
    if fmt == BF16:
        return {"k": junk(dim, torch.bfloat16, 2), "v": junk(dim, torch.bfloat16, 2), "ks": None, "vs": None}
    last, dt = (dim, torch.int8) if fmt == Q8_0 else (dim // 2, torch.uint8)
    return {"k": junk(last, dt, 1), "v": junk(last, dt, 1),
            "ks": junk(dim // 32, torch.float16, 2), "vs": junk(dim // 32, torch.float16, 2)}


def _fill(cache, name, pages, values, fmt):
    codes, scales = _encode(values, fmt)
    cache[name][pages] = codes
    if scales is not None:
        cache[name + "s"][pages] = scales


def _lengths(case):
    """Context and new tokens of each sequence; ragged: contexts down to a quarter, new tokens down to one."""
    c, B = case, case["batch"]
    if not c["ragged"]:
        return [c["ctx"]] * B, [c["tree"]] * B
    rng = random.Random(c["ctx"] * 64 + c["tree"])
    return ([c["ctx"]] + [rng.randint(c["ctx"] // 4, c["ctx"]) for _ in range(B - 1)],
            [c["tree"]] + [rng.randint(1, c["tree"]) for _ in range(B - 1)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c = case
    s = {"case": dict(c)}
    x = torch.float32 if c.get("x") == "f32" else torch.bfloat16
    if c["op"] == "rope":
        T, H, KV, D, P = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        # the three projections of a token beside each other, as a fused QKV product writes them
        rows = _normal(gen, (T, (H + 2 * KV) * D), x)
        s["q"] = rows[:, :H * D].unflatten(-1, (H, D))
        s["k"] = rows[:, H * D:(H + KV) * D].unflatten(-1, (KV, D))
        s["v"] = rows[:, (H + KV) * D:].unflatten(-1, (KV, D))
        s["gq"] = 1.0 + 0.1 * _normal(gen, (D,)) if c["norm"] else None
        s["gk"] = 1.0 + 0.1 * _normal(gen, (D,)) if c["norm"] else None
        # the rotation's table: cos and sin of position x frequency
        n_pos = c["start"] + T
        angle = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * \
            torch.pow(10000.0, -torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        n_pages = (T + P - 1) // P + 3
        order = torch.randperm(n_pages, generator=gen, device="cuda")
        i = torch.arange(T, device="cuda")
        if c["one_prompt"]:                     # consecutive positions on consecutive places of its pages
            s["pos"] = (i + c["start"]).to(torch.int32)
            slots = order[i // P] * P + i % P
        else:                                   # one token of each of T sequences
            s["pos"] = torch.randint(0, n_pos, (T,), generator=gen, device="cuda", dtype=torch.int32)
            slots = torch.randperm(n_pages * P, generator=gen, device="cuda")[:T]
        s["slots"] = torch.where(i >= T - c["pad"], torch.full_like(slots, -1), slots)   # padding is not stored
        s["cache"] = _empty_cache(gen, n_pages, KV, P, D, c["fmt"])
    elif c["op"] == "cache":
        T, R, KV, D, P = c["tokens"], c["read"], c["kv_heads"], c["dim"], c["page"]
        n_pages = (R + P - 1) // P + 2
        s["cache"] = _empty_cache(gen, n_pages, KV, P, D, c["fmt"])
        order = torch.randperm(n_pages, generator=gen, device="cuda")
        pages = order[:(R + P - 1) // P]
        for name in ("k", "v"):
            _fill(s["cache"], name, pages, _normal(gen, (len(pages), KV, P, D)), c["fmt"])
        i = torch.arange(R, device="cuda")
        s["slots"] = pages[i // P] * P + i % P                 # the sequence, oldest token first
        s["new"] = s["slots"][R - T:].contiguous()
        s["k"], s["v"] = _normal(gen, (T, KV, D), x), _normal(gen, (T, KV, D), x)
    else:
        B, H, KV, D, P, T = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["tree"]
        ctx, n = (torch.tensor(t, device="cuda") for t in _lengths(c))
        s["ctx"] = ctx.to(torch.int32)
        s["q_start"] = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)]).to(torch.int32)
        s["tokens"] = int(s["q_start"][-1])
        per = (c["ctx"] + T + P - 1) // P
        s["pages"] = torch.randperm(B * per + 2, generator=gen, device="cuda")[:B * per].view(B, per).to(torch.int32)
        s["cache"] = _empty_cache(gen, B * per + 2, KV, P, D, c["fmt"])
        for b in range(0, B, max(1, B // 4)):                  # a few pieces, to spare memory
            pages = s["pages"][b:b + max(1, B // 4)].reshape(-1).long()
            for name in ("k", "v"):
                _fill(s["cache"], name, pages, _normal(gen, (len(pages), KV, P, D)), c["fmt"])
        # places behind each sequence's last token keep what was there
        at = torch.arange(per * P, device="cuda").view(1, per, P).expand(B, per, P)
        dead = at >= (ctx + n)[:, None, None]
        for name in ("k", "v", "ks", "vs"):
            t = s["cache"][name]
            if t is not None:
                rows = t[s["pages"].long()]                    # [B, per, KV, P, last]
                raw = torch.randint(0, 256, (rows.numel() * rows.element_size(),), generator=gen, device="cuda",
                                    dtype=torch.uint8).view(rows.dtype).view(rows.shape)
                t[s["pages"].long()] = torch.where(dead[:, :, None, :, None], raw, rows)
        s["q"] = _normal(gen, (s["tokens"], H, D), torch.bfloat16, FRESH)
        s["scale"] = 1.0 / math.sqrt(D)
        s["mask"] = None
        if not c["causal"]:
            # each drafted token has one parent before it in its tree (or none: a child of the context), and sees
            # its ancestors and itself
            pick = torch.rand((B, T), generator=gen, device="cuda").cpu()
            sees = torch.zeros((B, T), dtype=torch.int64)
            for t in range(T):
                parent = (pick[:, t] * (t + 1)).long() - 1
                above = torch.where(parent < 0, torch.zeros_like(parent), sees.gather(1, parent.clamp(min=0)[:, None])[:, 0])
                bit = (1 << t) if t < 63 else -(1 << 63)
                sees[:, t] = above | bit
            token = torch.arange(s["tokens"], device="cuda")
            b = torch.searchsorted(s["q_start"].long(), token, right=True) - 1
            s["mask"] = sees.cuda()[b, token - s["q_start"].long()[b]].contiguous()
    return s


# --- the framework's calls -----------------------------------------------------------------------------------------
_FMT = {BF16: "BF16", Q8_0: "Q8_0", Q4_0: "Q4_0"}


def _own(s):
    import block_quantized_gemv_gb300 as bqg
    c = s["case"]
    if "handle" not in s:       # what a program keeps beside its cache
        t = s["cache"]
        s["handle"] = bqg.KVCache(getattr(bqg, _FMT[c["fmt"]]), t["k"], t["v"], t["ks"], t["vs"])
        if c["op"] == "attn":
            s["ws"] = bqg.tree_attention_workspace(s["handle"], c["heads"], c["batch"], c["tree"])
    if c["op"] == "rope":
        q = bqg.qk_norm_rope_kv_write(s["q"], s["k"], s["v"], s["slots"], s["handle"], s["pos"], s["table"],
                                      gamma_q=s["gq"], gamma_k=s["gk"], eps=EPS if c["norm"] else None,
                                      interleaved=c["interleaved"])
        k, v = bqg.kv_read(s["handle"], s["slots"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "cache":
        bqg.kv_write(s["k"], s["v"], s["new"], s["handle"])
        k, v = bqg.kv_read(s["handle"], s["slots"])
        return {"k": k, "v": v}
    return bqg.tree_attention(s["q"], s["handle"], s["pages"], s["ctx"], s["q_start"], c["tree"], mask=s["mask"],
                              scale=s["scale"], ws=s["ws"])


# --- the plain forms -----------------------------------------------------------------------------------------------
def _norm_rope(x, gain, norm, table, rot, interleaved):
    """fp32 [tokens, heads, dim]: the norm over each head, then the rotation of its first `rot` values."""
    if norm:
        mean = x.double().square().sum(-1, keepdim=True) / x.shape[-1]
        x = (x * (1.0 / torch.sqrt(mean + EPS)).float()) * gain
    c, s = table[:, None, :rot // 2], table[:, None, rot // 2:]
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), rest], -1)
    a, b = head[..., :rot // 2], head[..., rot // 2:]
    return torch.cat([a * c - b * s, a * s + b * c, rest], -1)


def _store(cache, name, slots, x, fmt):
    """Writes the tokens that have a slot into the cache; one without writes what the first one writes (it has a slot)."""
    codes, scales = _encode(x, fmt)
    page = cache[name].shape[2]
    keep = slots >= 0
    to = slots.clamp(min=0)
    for n, t in ((name, codes), (name + "s", scales)):
        if t is not None:
            cache[n].index_put_((torch.where(keep, to // page, to[0] // page)[:, None],
                                 torch.arange(t.shape[1], device=t.device)[None],
                                 torch.where(keep, to % page, to[0] % page)[:, None]),
                                torch.where(keep[:, None, None], t, t[:1]))


def _load(cache, name, slots, fmt):
    """The cache's values at `slots`, fp32 [tokens, heads, dim]; zeros where a slot is negative."""
    page = cache[name].shape[2]
    at = slots.clamp(min=0)
    scales = cache[name + "s"]
    v = _decode(cache[name][at // page, :, at % page],
                None if scales is None else scales[at // page, :, at % page], fmt)
    return torch.where((slots >= 0)[:, None, None], v, torch.zeros_like(v))


def _attend(s):
    c, cache = s["case"], s["cache"]
    B, H, KV, D, P, T = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["tree"]
    G, L = H // KV, c["ctx"] + T
    dev = s["q"].device
    start, ctx = s["q_start"].long(), s["ctx"].long()
    n = start[1:] - start[:-1]
    at = torch.arange(L, device=dev)
    page = s["pages"].long()[:, at // P]
    live = at[None] < (ctx + n)[:, None]                                     # [B, L]

    def values(name):
        scales = cache[name + "s"]
        v = _decode(cache[name][page, :, at % P], None if scales is None else scales[page, :, at % P], c["fmt"])
        v = torch.where(live[:, :, None, None], v, torch.zeros_like(v))      # [B, L, KV, D]
        return v.transpose(1, 2)

    t = torch.arange(T, device=dev)
    rows = (start[:-1, None] + t[None]).clamp(max=s["tokens"] - 1)           # [B, T]
    q = s["q"][rows].float().view(B, T, KV, G, D).permute(0, 2, 1, 3, 4).reshape(B, KV, T * G, D)
    scores = torch.matmul(q, values("k").transpose(2, 3)) * s["scale"]       # [B, KV, T G, L]
    draft = at[None] - ctx[:, None]                                          # place among the sequence's new tokens
    if s["mask"] is None:
        new = draft[:, None] <= t[None, :, None]
    else:
        new = ((s["mask"][rows][:, :, None] >> draft.clamp(0, 63)[:, None]) & 1) == 1
    sees = live[:, None] & ((draft < 0)[:, None] | new)                      # [B, T, L]
    sees = sees[:, None, :, None].expand(B, 1, T, G, L).reshape(B, 1, T * G, L)
    scores = scores.masked_fill(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values("v")) / torch.where(total == 0, torch.ones_like(total), total)
    out = out.view(B, KV, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    token = torch.arange(s["tokens"], device=dev)
    b = torch.searchsorted(start, token, right=True) - 1
    return out[b, token - start[b]].to(torch.bfloat16)


def run(state):
    if own:
        return _own(state)
    s = state
    c = s["case"]
    if c["op"] == "rope":
        table = s["table"][s["pos"].long()]
        q = _norm_rope(s["q"].float(), s["gq"], c["norm"], table, c["rot"], c["interleaved"])
        k = _norm_rope(s["k"].float(), s["gk"], c["norm"], table, c["rot"], c["interleaved"])
        _store(s["cache"], "k", s["slots"], k, c["fmt"])
        _store(s["cache"], "v", s["slots"], s["v"].float(), c["fmt"])
        return {"q": q.to(torch.bfloat16), "k": _load(s["cache"], "k", s["slots"], c["fmt"]).to(torch.bfloat16),
                "v": _load(s["cache"], "v", s["slots"], c["fmt"]).to(torch.bfloat16)}
    if c["op"] == "cache":
        _store(s["cache"], "k", s["new"], s["k"].float(), c["fmt"])
        _store(s["cache"], "v", s["new"], s["v"].float(), c["fmt"])
        return {"k": _load(s["cache"], "k", s["slots"], c["fmt"]).to(torch.bfloat16),
                "v": _load(s["cache"], "v", s["slots"], c["fmt"]).to(torch.bfloat16)}
    return _attend(s)


# --- what a pass cannot do without ---------------------------------------------------------------------------------
def _held(fmt, dim):
    """Bytes of one head's cached row."""
    return 2 * dim if fmt == BF16 else dim + dim // 16 if fmt == Q8_0 else dim // 2 + dim // 16


def work(case):
    c = case
    D, KV = c["dim"], c["kv_heads"]
    row = _held(c["fmt"], D)
    x = 4 if c.get("x") == "f32" else 2
    if c["op"] == "rope":
        T, H = c["tokens"], c["heads"]
        distinct = T if c["one_prompt"] else min(T, c["start"] + T)
        stored = T - c["pad"]
        return {"bytes": T * (H + 2 * KV) * D * x + distinct * c["rot"] * 4 + T * 12 + (2 * D * 4 if c["norm"] else 0) +
                T * H * D * 2 + 2 * stored * KV * row + 2 * T * KV * D * 2,
                "flops": T * (H + KV) * (3 * c["rot"] + (4 * D if c["norm"] else 0)) + 4 * T * KV * D}
    if c["op"] == "cache":
        T, R = c["tokens"], c["read"]
        return {"bytes": 2 * T * KV * D * x + (T + R) * 8 + 2 * T * KV * row + 2 * (R - T) * KV * row +
                2 * R * KV * D * 2, "flops": 4 * T * KV * D + 2 * R * KV * D}
    H = c["heads"]
    ctxs, news = _lengths(c)
    ctx, n = sum(ctxs), sum(news)
    # every new token sees its context, and at most the new ones up to itself
    pairs = sum(t * a + t * (t + 1) / 2 for a, t in zip(ctxs, news))
    return {"bytes": 2 * (ctx + n) * KV * row + 2 * n * H * D * 2 + (ctx + n) / c["page"] * 4 + (0 if c["causal"] else 8 * n),
            "flops": 4 * pairs * H * D}


# --- from the definitions, in 64 bits ------------------------------------------------------------------------------
def _rows64(cache, name, page, off, fmt):
    """fp64 [tokens, heads, dim] of the cache at (page, place) pairs."""
    raw = cache[name][page, :, off]
    if fmt == BF16:
        return raw.to(torch.float64)
    d = torch.repeat_interleave(cache[name + "s"][page, :, off].to(torch.float64), 32, dim=-1)
    if fmt == Q8_0:
        return raw.to(torch.float64) * d
    j = torch.arange(d.shape[-1], device=raw.device)
    byte = raw[..., (j // 32) * 16 + j % 16].to(torch.int64)
    return (((byte >> (4 * ((j % 32) // 16))) & 15) - 8).to(torch.float64) * d


def _kept64(x, fmt):
    """The values that a cache of `fmt` stands for once fp64 rows x are stored in it."""
    if fmt == BF16:
        return x.to(torch.bfloat16).to(torch.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    lo, hi = b.min(-1, keepdim=True).values, b.max(-1, keepdim=True).values
    if fmt == Q8_0:
        d = (torch.maximum(-lo, hi) / 127.0).to(torch.float16).to(torch.float64)
    else:
        j = torch.arange(32, device=x.device)
        m = torch.where(hi > -lo, hi, lo)
        both = hi == -lo                                         # the same magnitude twice: the first one's sign
        first_hi = torch.where(b == hi, j, 99).min(-1, keepdim=True).values
        first_lo = torch.where(b == lo, j, 99).min(-1, keepdim=True).values
        m = torch.where(both & (first_hi < first_lo), hi, m)
        d = (m / -8.0).to(torch.float16).to(torch.float64)
    r = b / torch.where(d == 0, torch.ones_like(d), d)
    whole = torch.where(r < 0, torch.ceil(r - 0.5), torch.floor(r + 0.5))
    whole = whole.clamp(-127, 127) if fmt == Q8_0 else whole.clamp(-8, 7)
    return (whole * d).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        rot, D = c["rot"], c["dim"]
        tab = s["table"].to(torch.float64)[s["pos"].long()]
        z = torch.complex(tab[:, :rot // 2], tab[:, rot // 2:])[:, None]
        got = {}
        for name, gain in (("q", s["gq"]), ("k", s["gk"])):
            x = s[name].to(torch.float64)
            if c["norm"]:
                x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(torch.float64)
            i = torch.arange(rot // 2, device=x.device)
            one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            turned = torch.complex(x[..., one], x[..., two]) * z
            y = x.clone()
            y[..., one], y[..., two] = turned.real, turned.imag
            got[name] = y
        stored = (s["slots"] >= 0).to(torch.float64)[:, None, None]
        return {"q": got["q"], "k": _kept64(got["k"], c["fmt"]) * stored,
                "v": _kept64(s["v"].to(torch.float64), c["fmt"]) * stored}
    if c["op"] == "cache":
        P, old, got = c["page"], s["slots"][:c["read"] - c["tokens"]], {}
        for name in ("k", "v"):
            got[name] = torch.cat([_rows64(s["cache"], name, old // P, old % P, c["fmt"]),
                                   _kept64(s[name].to(torch.float64), c["fmt"])])
        return got
    H, KV, P = c["heads"], c["kv_heads"], c["page"]
    G = H // KV
    out = torch.zeros(s["tokens"], H, c["dim"], dtype=torch.float64, device="cuda")
    starts, ctxs = s["q_start"].tolist(), s["ctx"].tolist()
    for b in range(c["batch"]):
        q0, q1, ctx = starts[b], starts[b + 1], ctxs[b]
        n = q1 - q0
        at = torch.arange(ctx + n, device="cuda")
        page = s["pages"][b].long()[at // P]
        k = _rows64(s["cache"], "k", page, at % P, c["fmt"])
        v = _rows64(s["cache"], "v", page, at % P, c["fmt"])
        ok = torch.ones(n, ctx + n, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            ok[:, ctx:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            ok[:, ctx:] = (torch.bitwise_right_shift(s["mask"][q0:q1, None], torch.arange(n, device="cuda")) & 1).bool()
        for h in range(KV):
            qh = s["q"][q0:q1, h * G:(h + 1) * G].to(torch.float64)          # [n, G, D]
            a = torch.einsum("ngd,ld->ngl", qh, k[:, h]) * s["scale"]
            a = torch.where(ok[:, None], a, torch.full_like(a, -math.inf))
            out[q0:q1, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", torch.softmax(a, -1), v[:, h])
    return out
