"""What a speculative serving step needs around attention on a paged cache: cases, inputs and plain forms.

Four operators:

  share    Attention of each sequence's newest tokens where sequences share their first tokens (one prompt, sampled or
           branched many times): the shared part is read and multiplied once for all of its sequences.
  verify   Drafted tokens accepted or rejected against the target's probabilities, from given random numbers, and the
           token that follows: a chain or a tree of drafts, sampled ones (with the draft's probabilities) or chosen ones.
  compact  The accepted path's keys and values moved to the places behind each sequence's context.
  fork     Sequences branched: a branch shares its parent's full pages and gets a copy of the page in use.

The cache is n_pages pages of `page` tokens for each KV head.  bf16: values.  q8_0: int8 codes and one fp16 scale
per 32 values, value q d.  q4_0: two codes per byte (element j low, j + 16 high, within 32), value (q - 8) d.

Verification, per sequence: token 0 is the last one given out, each other one i has a parent before it.  p is the
target's distribution after a token, q the draft's.  At a token, its drafts are taken in their order; draft t is accepted
when u q(t) Z < r(t), where r = p and Z = 1 before the first rejection.  A rejection makes r(x) = max(p(x) - c q(x), 0)
with c the sum of the Z so far, and Z the sum of the new r.  With all rejected, or none there, the next token is the first
one at which the running sum of r exceeds u' times the whole (u': the number of token 0), r = p if nothing is left of
it.  Chosen drafts have q = 1 at their token: r is p without the rejected tokens and Z = 1 - their p.
"""
import math
import random

import torch

own = False

BF16, Q8_0, Q4_0 = "bf16", "q8_0", "q4_0"
FRESH = 1.5     # spread of the attention's queries: scores of a few units, some keys stand out


# --- cases ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # four samples of one chat of an 8B-style model (32 query heads on 8 KV heads): latency counts
        dict(name="share 4x(1000+77) q8_0", op="share", fmt=Q8_0, groups=1, per=4, prefix=1000, ctx=77, tree=1,
             ragged=False, heads=32, kv_heads=8, dim=128, page=64, causal=True),
        # a serving batch behind one long system prompt, one token each
        dict(name="share 64x(8192+500) bf16", op="share", fmt=BF16, groups=1, per=64, prefix=8192, ctx=500, tree=1,
             ragged=True, heads=32, kv_heads=8, dim=128, page=64, causal=True),
        # several prompts, each sampled many times, no shared heads, small pages
        dict(name="share 6x16x(2999+300) mha q4_0", op="share", fmt=Q4_0, groups=6, per=16, prefix=2999, ctx=300, tree=1,
             ragged=True, heads=32, kv_heads=32, dim=128, page=16, causal=True),
        # drafted trees behind a long shared document
        dict(name="share 8x(32768+900) tree 13 q8_0", op="share", fmt=Q8_0, groups=1, per=8, prefix=32768, ctx=900,
             tree=13, ragged=True, heads=32, kv_heads=8, dim=128, page=128, causal=False),
        # a wide batch of a 70B-style model with short drafted chains: bound by the products
        dict(name="share 96x(16384+400) chain 4 bf16", op="share", fmt=BF16, groups=1, per=96, prefix=16384, ctx=400,
             tree=4, ragged=False, heads=64, kv_heads=8, dim=128, page=64, causal=True),
        # one chat, a chain of five sampled drafts, a small vocabulary: latency counts
        dict(name="verify 1 chain 6 of 32000", op="verify", batch=1, tree=6, vocab=32000, x="f32", drafted=True,
             chain=True, ragged=False),
        # a batch with chosen trees of an odd vocabulary, probabilities in bf16
        dict(name="verify 16 trees 24 of 100003 bf16", op="verify", batch=16, tree=24, vocab=100003, x="bf16",
             drafted=False, chain=False, ragged=True),
        # a wide batch with sampled trees
        dict(name="verify 64 trees 10 of 131072", op="verify", batch=64, tree=10, vocab=131072, x="f32", drafted=True,
             chain=False, ragged=True),
        # the accepted path of one chat: latency counts
        dict(name="compact 1x13 q8_0", op="compact", batch=1, tree=13, ctx=4095, fmt=Q8_0, kv_heads=8, dim=128, page=64),
        # a wide batch with large trees, no shared heads, small pages
        dict(name="compact 64x64 bf16", op="compact", batch=64, tree=64, ctx=1000, fmt=BF16, kv_heads=32, dim=128,
             page=16),
        # one chat branched four ways
        dict(name="fork 1x4 of 777 q8_0", op="fork", parents=1, per=4, ctx=777, fmt=Q8_0, kv_heads=8, dim=128, page=64),
        # a batch of prompts, each sampled 16 times
        dict(name="fork 32x16 of 5000 q4_0", op="fork", parents=32, per=16, ctx=5000, fmt=Q4_0, kv_heads=8, dim=128,
             page=128),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["share", "share", "verify", "verify", "compact", "fork"])
    fmt = rng.choice([BF16, Q8_0, Q4_0])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    if op == "share":
        heads = kv * rng.choice([g for g in (1, 2, 3, 4, 4, 5, 7, 8, 16) if kv * g <= 64])
        causal = rng.random() < 0.5
        tree = rng.choice([1, 1, _log(rng, 1, 64)]) if causal else _log(rng, 2, 64)
        groups = rng.choice([1, 1, 1, _log(rng, 2, 12)])
        per = _log(rng, 1, max(1, min(128, 1024 // (groups * tree))))
        n = groups * per
        # own tokens, then shared ones: at most about the bytes and the products of the largest listed case
        ctx = _log(rng, 1, max(1, min(80_000_000 // (n * kv * dim), 4_000_000_000 // (n * heads * tree * dim), 8000))) - 1
        room = min(60_000_000 // (groups * kv * dim), 40_000_000_000 // (n * heads * tree * dim), 65000)
        return dict(op=op, fmt=fmt, groups=groups, per=per, prefix=_log(rng, 1, max(1, room)), ctx=ctx, tree=tree,
                    ragged=rng.random() < 0.6, heads=heads, kv_heads=kv, dim=dim, page=page, causal=causal)
    if op == "verify":
        vocab = _log(rng, 100, 262144)
        tree = _log(rng, 1, 64)
        batch = _log(rng, 1, max(1, min(128, 64 * 10 * 131072 // (vocab * tree))))
        return dict(op=op, batch=batch, tree=tree, vocab=vocab, x=rng.choice(["f32", "bf16"]),
                    drafted=rng.random() < 0.6, chain=rng.random() < 0.4, ragged=rng.random() < 0.6)
    if op == "compact":
        tree = _log(rng, 1, 64)
        batch = _log(rng, 1, max(1, min(256, 64 * 64 * 32 * 128 // (tree * kv * dim))))
        ctx = _log(rng, 1, max(1, min(3000, 280_000_000 // (batch * kv * dim)))) - 1
        return dict(op=op, batch=batch, tree=tree, ctx=ctx, fmt=fmt, kv_heads=kv, dim=dim, page=page)
    per = _log(rng, 1, 64)
    parents = _log(rng, 1, max(1, min(64, 32 * 16 * 64 * 8 * 128 // (per * page * kv * dim))))
    ctx = _log(rng, 1, max(1, min(6000, 200_000_000 // (parents * kv * dim))))
    return dict(op=op, parents=parents, per=per, ctx=ctx, fmt=fmt, kv_heads=kv, dim=dim, page=page)


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
        d = (b.abs().amax(-1, keepdim=True) / 127.0).half()
        q = _away(b / torch.where(d == 0, torch.ones_like(d), d).float())
        return q.clamp(-127, 127).to(torch.int8).flatten(-2), d.squeeze(-1)
    m = b.gather(-1, b.abs().argmax(-1, keepdim=True))
    d = (m / -8.0).half()
    q = (_away(b / torch.where(d == 0, torch.ones_like(d), d).float()) + 8).clamp(0, 15).to(torch.uint8)
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


def _cache(gen, n_pages, kv, page, dim, fmt):
    """A cache whose every page holds keys and values."""
    c = {"k": [], "v": [], "ks": [], "vs": []}
    step = max(1, (1 << 26) // (kv * page * dim))              # a few pieces, to spare memory
    for p in range(0, n_pages, step):
        for name in ("k", "v"):
            codes, scales = _encode(_normal(gen, (min(step, n_pages - p), kv, page, dim)), fmt)
            c[name].append(codes)
            if scales is not None:
                c[name + "s"].append(scales)
    return {name: torch.cat(t) if t else None for name, t in c.items()}


def _spread(rng, most, n, least=0):
    """`most`, then n - 1 whole numbers from a quarter of it on."""
    return [most] + [rng.randint(max(least, most // 4), most) for _ in range(n - 1)]


def _lengths(case):
    """share: tokens of each prefix, own ones and new ones of each sequence."""
    c, G, n = case, case["groups"], case["groups"] * case["per"]
    if not c["ragged"]:
        return [c["prefix"]] * G, [c["ctx"]] * n, [c["tree"]] * n
    rng = random.Random(c["prefix"] * 64 + c["tree"])
    return _spread(rng, c["prefix"], G), _spread(rng, c["ctx"], n), _spread(rng, c["tree"], n, 1)


def _paths(case):
    """compact: the accepted path of each sequence: places among its new tokens, ascending from 0."""
    rng = random.Random(case["ctx"] * 64 + case["tree"])
    T, out = case["tree"], []
    for _ in range(case["batch"]):
        n = rng.randint(1, max(1, (T + 1) // 2))
        out.append([0] + sorted(rng.sample(range(1, T), min(n, T) - 1)) if T > 1 else [0])
    return out


def _forks(case):
    """fork: the tokens of each parent."""
    return _spread(random.Random(case["ctx"]), case["ctx"], case["parents"], 1)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _prepare_share(s, gen):
    c = s["case"]
    G, per, H, KV, D, P = c["groups"], c["per"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    prefix, own_ctx, new = _lengths(c)
    n = G * per
    s["prefix_len"] = _ints(prefix)
    s["seq_start"] = _ints([g * per for g in range(G + 1)])
    s["ctx"] = _ints([prefix[i // per] + own_ctx[i] for i in range(n)])
    start = [0]
    for t in new:
        start.append(start[-1] + t)
    s["q_start"], s["tokens"] = _ints(start), start[-1]
    # as forks leave them: a prefix's full pages are shared, its last, partly filled one has a copy in each sequence
    most = max((prefix[i // per] + own_ctx[i] + new[i] + P - 1) // P for i in range(n))
    total = sum(p // P for p in prefix) + sum(
        (prefix[i // per] + own_ctx[i] + new[i] + P - 1) // P - prefix[i // per] // P for i in range(n)) + 2
    order = torch.randperm(total, generator=gen, device="cuda").tolist()
    s["cache"] = _cache(gen, total, KV, P, D, c["fmt"])
    rows, copies, at = [], [], 0
    for g in range(G):
        full = prefix[g] // P
        shared, at = order[at:at + full], at + full
        first = None
        for i in range(g * per, (g + 1) * per):
            k = (prefix[g] + own_ctx[i] + new[i] + P - 1) // P - full
            mine, at = order[at:at + k], at + k
            if first is None:
                first = mine[0]
            else:
                copies.append((first, mine[0], prefix[g] % P))
            rows.append((shared + mine + [0] * most)[:most])
    s["pages"] = _ints(rows)
    if copies:
        a, b, used = _ints(copies, torch.long).unbind(1)
        keep = torch.arange(P, device="cuda")[None, None, :, None] < used[:, None, None, None]
        for t in s["cache"].values():
            if t is not None:
                t[b] = torch.where(keep, t[a], t[b])
    s["q"] = _normal(gen, (s["tokens"], H, D), torch.bfloat16, FRESH)
    s["scale"] = 1.0 / math.sqrt(D)
    s["mask"] = None
    if not c["causal"]:
        # each drafted token has one parent before it in its tree (or none: a child of the context), and sees
        # its ancestors and itself
        T = c["tree"]
        pick = torch.rand((n, T), generator=gen, device="cuda").cpu()
        sees = torch.zeros((n, T), dtype=torch.int64)
        for t in range(T):
            parent = (pick[:, t] * (t + 1)).long() - 1
            above = torch.where(parent < 0, torch.zeros_like(parent), sees.gather(1, parent.clamp(min=0)[:, None])[:, 0])
            sees[:, t] = above | ((1 << t) if t < 63 else -(1 << 63))
        token = torch.arange(s["tokens"], device="cuda")
        b = torch.searchsorted(s["q_start"].long(), token, right=True) - 1
        s["mask"] = sees.cuda()[b, token - s["q_start"].long()[b]].contiguous()


def _prepare_verify(s, gen):
    c = s["case"]
    B, T, V = c["batch"], c["tree"], c["vocab"]
    dtype = torch.float32 if c["x"] == "f32" else torch.bfloat16
    rng = random.Random(V * 64 + T)
    new = _spread(rng, T, B, 1) if c["ragged"] else [T] * B
    start = [0]
    for t in new:
        start.append(start[-1] + t)
    n = start[-1]
    s["q_start"] = _ints(start)
    s["u"] = torch.rand(n, generator=gen, device="cuda")
    # a parent before each token; trees are bushy at their beginnings
    pick = torch.rand(n, generator=gen, device="cuda").tolist()
    parent = [(i - 1 if c["chain"] else int(pick[start[b] + i] ** 2 * i)) if i else -1
              for b in range(B) for i in range(new[b])]
    s["parent"] = _ints(parent)
    first = [start[b] for b in range(B) for _ in range(new[b])]
    row = _ints([f + max(p, 0) for f, p in zip(first, parent)], torch.long)      # of each token's parent
    nth, seen = [], {}
    for r, p in zip(row.tolist(), parent):                                       # how many-th child it is
        nth.append(seen.get(r, 0) if p >= 0 else 0)
        if p >= 0:
            seen[r] = nth[-1] + 1
    target = torch.empty((n, V), dtype=dtype, device="cuda")
    draft = torch.empty((n, V), dtype=dtype, device="cuda") if c["drafted"] else None
    best = min(V, max(nth) + 1)
    top = torch.empty((n, best), dtype=torch.long, device="cuda")
    step = max(1, (1 << 26) // V)
    for i in range(0, n, step):
        # a model's next-token distribution: a few likely tokens over a long tail; the draft's is near it
        x = _normal(gen, (min(step, n - i), V), scale=3.0)
        y = x + _normal(gen, x.shape, scale=0.6)
        target[i:i + step] = torch.softmax(x, -1).to(dtype)
        if draft is not None:
            draft[i:i + step] = torch.softmax(y, -1).to(dtype)
        else:
            top[i:i + step] = y.topk(best, -1).indices
    s["target"], s["draft"] = target, draft
    if draft is not None:                                       # sampled from the parent's distribution
        tokens = torch.empty(n, dtype=torch.long, device="cuda")
        for i in range(0, n, step):
            tokens[i:i + step] = torch.multinomial(draft[row[i:i + step]].float(), 1, generator=gen)[:, 0]
    else:                                                       # its likeliest, one after the other
        tokens = top[row, _ints(nth, torch.long)]
    s["tokens"] = tokens.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c = case
    s = {"case": dict(c)}
    if c["op"] == "share":
        _prepare_share(s, gen)
    elif c["op"] == "verify":
        _prepare_verify(s, gen)
    elif c["op"] == "compact":
        B, T, P = c["batch"], c["tree"], c["page"]
        per = (c["ctx"] + T + P - 1) // P
        total = B * per + 2
        s["cache"] = _cache(gen, total, c["kv_heads"], P, c["dim"], c["fmt"])
        s["pages"] = torch.randperm(total, generator=gen, device="cuda")[:B * per].view(B, per).to(torch.int32)
        ctx = [c["ctx"] - (b % (c["ctx"] // 4 + 1)) for b in range(B)]
        s["ctx"] = _ints(ctx)
        paths = _paths(c)
        s["path"] = _ints([p + [-1] * (T - len(p)) for p in paths])
        s["n_path"] = _ints([len(p) for p in paths])
        b = _ints([b for b in range(B) for _ in paths[b]], torch.long)
        to = _ints([ctx[b] + k for b in range(B) for k in range(len(paths[b]))], torch.long)
        s["kept"] = s["pages"][b, to // P].long() * P + to % P             # where the kept tokens are afterwards
    else:
        N, per, P = c["parents"], c["per"], c["page"]
        ctx = _forks(c)
        wide = max(ctx) // P + 2
        total = N * wide + N * per + 2
        order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        s["cache"] = _cache(gen, total, c["kv_heads"], P, c["dim"], c["fmt"])
        # the parents' rows, then free ones
        s["pages"] = torch.full((N * (per + 1), wide), -1, dtype=torch.int32, device="cuda")
        used = _ints([x // P + 1 for x in ctx])
        s["pages"][:N] = torch.where(torch.arange(wide, device="cuda")[None] < used[:, None], order[:N * wide].view(N, wide),
                                     torch.full_like(s["pages"][:N], -1))
        s["ctx"] = _ints(ctx + [0] * (N * per))
        s["parent"] = _ints([i for i in range(N) for _ in range(per)])
        s["child"] = _ints([N + i for i in range(N * per)])
        s["fresh"] = order[N * wide:N * wide + N * per].contiguous()
        n = _ints([x % P for x in ctx for _ in range(per)], torch.long)
        at = torch.arange(P, device="cuda")[None].expand(N * per, P)
        s["copied"] = (s["fresh"].long()[:, None] * P + at)[at < n[:, None]]       # slots of the copied tokens
    return s


# --- the framework's calls -----------------------------------------------------------------------------------------
_FMT = {BF16: "BF16", Q8_0: "Q8_0", Q4_0: "Q4_0"}


def _own(s):
    import block_quantized_gemv_gb300 as bqg
    c = s["case"]
    if c["op"] == "verify":
        accepted, path, token = bqg.tree_verify(s["target"], s["tokens"], s["q_start"], c["tree"], s["u"],
                                                parent=None if c["chain"] else s["parent"], draft=s["draft"])
        return {"accepted": accepted, "path": path, "token": token}
    if "handle" not in s:       # what a program keeps beside its cache
        t = s["cache"]
        s["handle"] = bqg.KVCache(getattr(bqg, _FMT[c["fmt"]]), t["k"], t["v"], t["ks"], t["vs"])
        if c["op"] == "share":
            s["ws"] = bqg.shared_prefix_attention_workspace(s["handle"], c["heads"], c["groups"] * c["per"], c["tree"],
                                                            s["tokens"], c["groups"])
    if c["op"] == "share":
        return bqg.shared_prefix_attention(s["q"], s["handle"], s["pages"], s["ctx"], s["q_start"], c["tree"],
                                           s["prefix_len"], s["seq_start"], mask=s["mask"], scale=s["scale"], ws=s["ws"])
    if c["op"] == "compact":
        ctx = bqg.kv_compact(s["handle"], s["pages"], s["ctx"], s["path"], s["n_path"])
        k, v = bqg.kv_read(s["handle"], s["kept"])
        return {"ctx": ctx, "k": k, "v": v}
    bqg.kv_fork(s["handle"], s["pages"], s["ctx"], s["parent"], s["child"], s["fresh"])
    k, v = bqg.kv_read(s["handle"], s["copied"])
    return {"pages": s["pages"], "ctx": s["ctx"], "k": k, "v": v}


# --- the plain forms -----------------------------------------------------------------------------------------------
def _load(cache, name, slots, fmt):
    """The cache's values at `slots`, fp32 [tokens, heads, dim]."""
    page = cache[name].shape[2]
    scales = cache[name + "s"]
    return _decode(cache[name][slots // page, :, slots % page],
                   None if scales is None else scales[slots // page, :, slots % page], fmt)


def _share(s):
    c, cache = s["case"], s["cache"]
    G, per, H, KV, D, P, T = c["groups"], c["per"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["tree"]
    n, R = G * per, H // KV
    dev = s["q"].device
    start, ctx, prefix = s["q_start"].long(), s["ctx"].long(), s["prefix_len"].long()
    new = start[1:] - start[:-1]
    head = torch.repeat_interleave(prefix, per, output_size=n)                # shared tokens of each sequence
    L = c["prefix"], c["ctx"] + T                                             # shared ones, own ones at most
    wide = s["pages"].shape[1] * P - 1

    def values(name, pages, at, live):                                        # pages [b, .], at [b, l] -> [b, KV, l, D]
        at = at.clamp(max=wide)
        page = pages.long().gather(1, at // P)
        scales = cache[name + "s"]
        v = _decode(cache[name][page, :, at % P], None if scales is None else scales[page, :, at % P], c["fmt"])
        return torch.where(live[:, :, None, None], v, torch.zeros_like(v)).transpose(1, 2)

    t = torch.arange(T, device=dev)
    rows = (start[:-1, None] + t[None]).clamp(max=s["tokens"] - 1)            # [n, T]
    q = s["q"][rows].float().view(n, T, KV, R, D).permute(0, 2, 1, 3, 4)      # [n, KV, T, R, D]
    # the shared tokens: all rows of a prefix at once
    at = torch.arange(L[0], device=dev)[None].expand(G, L[0])
    live = at < prefix[:, None]
    pages = s["pages"][s["seq_start"][:-1].long()]
    qs = q.reshape(G, per, KV, T * R, D).transpose(1, 2).reshape(G, KV, per * T * R, D)
    a = torch.matmul(qs, values("k", pages, at, live).transpose(2, 3)) * s["scale"]
    a = a.masked_fill(~live[:, None, None], -math.inf)
    # the own ones
    at2 = head[:, None] + torch.arange(L[1], device=dev)[None]
    live2 = at2 < (ctx + new)[:, None]
    b = torch.matmul(q.reshape(n, KV, T * R, D), values("k", s["pages"], at2, live2).transpose(2, 3)) * s["scale"]
    draft = at2 - ctx[:, None]                                                # place among the sequence's new tokens
    if s["mask"] is None:
        fresh = draft[:, None] <= t[None, :, None]
    else:
        fresh = ((s["mask"][rows][:, :, None] >> draft.clamp(0, 63)[:, None]) & 1) == 1
    sees = live2[:, None] & ((draft < 0)[:, None] | fresh)                    # [n, T, l]
    b = b.masked_fill(~sees[:, None, :, None].expand(n, 1, T, R, L[1]).reshape(n, 1, T * R, L[1]), -math.inf)
    top = b.amax(-1, keepdim=True)
    first = a.amax(-1, keepdim=True).view(G, KV, per, T * R, 1).transpose(1, 2).reshape(n, KV, T * R, 1)
    top = torch.maximum(top, first)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    top_a = top.view(G, per, KV, T * R, 1).transpose(1, 2).reshape(G, KV, per * T * R, 1)
    a, b = torch.exp(a - top_a), torch.exp(b - top)

    def rows_of(x):
        return x.view(G, KV, per, T * R, -1).transpose(1, 2).reshape(n, KV, T * R, -1)

    total = rows_of(a.sum(-1, keepdim=True)) + b.sum(-1, keepdim=True)
    out = rows_of(torch.matmul(a, values("v", pages, at, live))) + torch.matmul(b, values("v", s["pages"], at2, live2))
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    out = out.view(n, KV, T, R, D).permute(0, 2, 1, 3, 4).reshape(n, T, H, D)
    token = torch.arange(s["tokens"], device=dev)
    i = torch.searchsorted(start, token, right=True) - 1
    return out[i, token - start[i]].to(torch.bfloat16)


def _verify(s):
    """All sequences at once, one place of their trees after the other: a token's drafts stand behind it in their order."""
    c = s["case"]
    B, T, V = c["batch"], c["tree"], c["vocab"]
    dev = s["u"].device
    start = s["q_start"].long()
    new = start[1:] - start[:-1]
    zero = torch.zeros(B, dtype=torch.long, device=dev)
    node, count = zero, zero + 1
    path = torch.full((B, T), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    Z = torch.ones(B, dtype=torch.float64, device=dev)         # sum of what is left at the node; c: what is taken off
    taken = torch.zeros(B, dtype=torch.float64, device=dev)
    gone = torch.zeros((B, T), dtype=torch.long, device=dev)   # chosen drafts rejected at the node (place 0: none)
    lane = torch.arange(B, device=dev)
    for i in range(1, T):
        here = (start[:-1] + i).clamp(max=s["u"].numel() - 1)
        up = zero + i - 1 if c["chain"] else s["parent"][here].long()
        asked = (i < new) & (up == node)
        row, tok, u = start[:-1] + node, s["tokens"][here].long(), s["u"][here].double()
        p = s["target"][row, tok].double()
        if s["draft"] is not None:
            q = s["draft"][row, tok].double()
            yes = asked & (u * q * Z < (p - taken * q).clamp(min=0))
        else:
            again = ((gone > 0) & (s["tokens"][(start[:-1, None] + gone).clamp(max=s["u"].numel() - 1)].long() ==
                                   tok[:, None])).any(-1)
            p = torch.where(again, torch.zeros_like(p), p)
            yes = asked & (u * Z < p)
        no = asked & ~yes
        if s["draft"] is not None:
            taken = torch.where(no, taken + Z, taken)
            rest = s["target"][row].double() - taken[:, None] * s["draft"][row].double()
            Z = torch.where(no, rest.clamp(min=0).sum(-1), Z)
        else:
            Z = torch.where(no, Z - p, Z)
            gone[:, i] = torch.where(no, zero + i, zero)
        node = torch.where(yes, zero + i, node)
        Z = torch.where(yes, torch.ones_like(Z), Z)
        taken = torch.where(yes, torch.zeros_like(taken), taken)
        gone = torch.where(yes[:, None], torch.zeros_like(gone), gone)
        path[lane, torch.where(yes, count, zero)] = torch.where(yes, i, path[:, 0])
        count = count + yes
    row = start[:-1] + node
    p = s["target"][row].double()
    if s["draft"] is not None:
        r = (p - taken[:, None] * s["draft"][row].double()).clamp(min=0)
        r = torch.where((taken > 0)[:, None], r, p)
    else:
        at = s["tokens"][(start[:-1, None] + gone).clamp(max=s["u"].numel() - 1)].long()
        r = p.scatter_reduce(1, at, torch.where(gone > 0, torch.zeros_like(at, dtype=p.dtype), p.gather(1, at)), "amin")
    left = r.sum(-1, keepdim=True)
    r = torch.where(left > 0, r, p)
    run_sum = r.cumsum(-1)
    past = run_sum > s["u"][start[:-1]].double()[:, None] * run_sum[:, -1:]
    token = torch.where(past, torch.arange(V, device=dev)[None], V - 1).amin(-1)
    return {"accepted": count.to(torch.int32), "path": path, "token": token.to(torch.int32)}


def _move(s, src, dst):
    """Cached tokens at slots src to slots dst; all are read before any is written."""
    for t in s["cache"].values():
        if t is not None:
            P = t.shape[2]
            t[dst // P, :, dst % P] = t[src // P, :, src % P]


def run(state):
    if own:
        return _own(state)
    s = state
    c = s["case"]
    if c["op"] == "share":
        return _share(s)
    if c["op"] == "verify":
        return _verify(s)
    P = c["page"]
    if c["op"] == "compact":
        k = torch.arange(c["tree"], device=s["ctx"].device)[None]
        live = k < s["n_path"][:, None]
        # places without a token stay where they are
        ctx = s["ctx"].long()[:, None]
        src, dst = ctx + torch.where(live, s["path"].long(), k), ctx + k
        pages = s["pages"].long()
        _move(s, (pages.gather(1, src // P) * P + src % P).flatten(), (pages.gather(1, dst // P) * P + dst % P).flatten())
        return {"ctx": s["ctx"] + s["n_path"], "k": _load(s["cache"], "k", s["kept"], c["fmt"]).to(torch.bfloat16),
                "v": _load(s["cache"], "v", s["kept"], c["fmt"]).to(torch.bfloat16)}
    up, child, fresh = s["parent"].long(), s["child"].long(), s["fresh"].long()
    ctx = s["ctx"].long()[up]
    full = ctx // P
    old = s["pages"].long()[up].gather(1, full[:, None])[:, 0]
    column = torch.arange(s["pages"].shape[1], device=ctx.device)[None]
    rows = torch.where(column < full[:, None], s["pages"][up], s["pages"][child])
    s["pages"][child] = torch.where(column == full[:, None], s["fresh"][:, None], rows)
    s["ctx"][child] = s["ctx"][up]
    used = (torch.arange(P, device=ctx.device)[None] < (ctx % P)[:, None])[:, None, :, None]
    for t in s["cache"].values():
        if t is not None:
            t[fresh] = torch.where(used, t[old], t[fresh])
    return {"pages": s["pages"], "ctx": s["ctx"], "k": _load(s["cache"], "k", s["copied"], c["fmt"]).to(torch.bfloat16),
            "v": _load(s["cache"], "v", s["copied"], c["fmt"]).to(torch.bfloat16)}


# --- what a pass cannot do without ---------------------------------------------------------------------------------
def _held(fmt, dim):
    """Bytes of one head's cached row."""
    return 2 * dim if fmt == BF16 else dim + dim // 16 if fmt == Q8_0 else dim // 2 + dim // 16


def work(case):
    c = case
    if c["op"] == "verify":
        # the numbers that decide, and the row (with chosen drafts one, with sampled ones two) that the last draw is from
        rows = c["batch"] * (2 if c["drafted"] else 1)
        size = 4 if c["x"] == "f32" else 2
        return {"bytes": rows * c["vocab"] * size + c["batch"] * c["tree"] * 20, "flops": rows * c["vocab"] * 2}
    D, KV = c["dim"], c["kv_heads"]
    row = _held(c["fmt"], D)
    if c["op"] == "share":
        prefix, own_ctx, new = _lengths(c)
        H, per = c["heads"], c["per"]
        pairs = sum(t * (prefix[i // per] + own_ctx[i]) + t * (t + 1) / 2 for i, t in enumerate(new))
        return {"bytes": 2 * (sum(prefix) + sum(own_ctx) + sum(new)) * KV * row + 2 * sum(new) * H * D * 2,
                "flops": 4 * pairs * H * D}
    if c["op"] == "compact":
        paths = _paths(c)
        moved = sum(k != j for p in paths for k, j in enumerate(p))
        kept = sum(len(p) for p in paths)
        return {"bytes": 4 * moved * KV * row + 2 * (kept - moved) * KV * row + 2 * kept * KV * D * 2 + kept * 12,
                "flops": 2 * kept * KV * D}
    P, ctx = c["page"], _forks(c)
    copied = c["per"] * sum(x % P for x in ctx)
    table = sum(x // P * 4 for x in ctx)
    return {"bytes": 2 * sum(x % P for x in ctx) * KV * row + 2 * copied * KV * row + 2 * copied * KV * D * 2 + copied * 8 +
            table * (c["per"] + 1), "flops": 2 * copied * KV * D}


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


def _verify64(s):
    c = s["case"]
    starts, tokens, u = s["q_start"].tolist(), s["tokens"].tolist(), s["u"].tolist()
    parent = s["parent"].tolist()
    accepted, paths, last = [], [], []
    for b in range(c["batch"]):
        q0, n = starts[b], starts[b + 1] - starts[b]
        node, path = 0, [0]
        while True:
            p = s["target"][q0 + node].to(torch.float64)
            q = None if s["draft"] is None else s["draft"][q0 + node].to(torch.float64)
            r, Z, c_off, found = p.clone(), 1.0, 0.0, -1
            for i in range(node + 1, n):
                if (i - 1 if c["chain"] else parent[q0 + i]) != node:
                    continue
                t = tokens[q0 + i]
                if u[q0 + i] * (1.0 if q is None else float(q[t])) * Z < float(r[t]):
                    found = i
                    break
                if q is None:
                    Z -= float(r[t])
                    r[t] = 0.0
                else:
                    c_off += Z
                    r = torch.relu(p - c_off * q)
                    Z = float(r.sum())
            if found < 0:
                break
            node = found
            path.append(node)
        if float(r.sum()) <= 0.0:
            r = p
        run_sum = torch.cumsum(r, 0)
        hit = torch.nonzero(run_sum > u[q0] * float(run_sum[-1]))
        last.append(int(hit[0]))
        accepted.append(len(path))
        paths.append(path + [-1] * (c["tree"] - len(path)))
    return {"accepted": _ints(accepted), "path": _ints(paths), "token": _ints(last)}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "verify":
        return _verify64(s)
    P = c["page"]
    if c["op"] == "compact":
        ctx, at, paths = s["ctx"].tolist(), [], _paths(c)
        for b, path in enumerate(paths):
            at += [(b, ctx[b] + j) for j in path]
        b, tok = (torch.tensor(x, device="cuda") for x in zip(*at))
        page = s["pages"].long()[b, tok // P]
        return {"ctx": s["ctx"] + s["n_path"], "k": _rows64(s["cache"], "k", page, tok % P, c["fmt"]),
                "v": _rows64(s["cache"], "v", page, tok % P, c["fmt"])}
    if c["op"] == "fork":
        pages, ctx, page, off = s["pages"].clone(), s["ctx"].clone(), [], []
        for up, child, fresh in zip(s["parent"].tolist(), s["child"].tolist(), s["fresh"].tolist()):
            n = int(ctx[up])
            pages[child, :n // P] = pages[up, :n // P]
            pages[child, n // P] = fresh
            ctx[child] = n
            page += [int(pages[up, n // P])] * (n % P)
            off += range(n % P)
        page, off = torch.tensor(page, dtype=torch.long, device="cuda"), torch.tensor(off, dtype=torch.long, device="cuda")
        return {"pages": pages, "ctx": ctx, "k": _rows64(s["cache"], "k", page, off, c["fmt"]),
                "v": _rows64(s["cache"], "v", page, off, c["fmt"])}
    H, KV = c["heads"], c["kv_heads"]
    G = H // KV
    out = torch.zeros(s["tokens"], H, c["dim"], dtype=torch.float64, device="cuda")
    starts, ctxs = s["q_start"].tolist(), s["ctx"].tolist()
    for b in range(c["groups"] * c["per"]):
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
        q = s["q"][q0:q1].to(torch.float64).view(n, KV, G, -1)
        a = torch.einsum("nhgd,lhd->nhgl", q, k) * s["scale"]
        a = torch.where(ok[:, None, None], a, torch.full_like(a, -math.inf))
        out[q0:q1] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(a, -1), v).reshape(n, H, -1)
    return out
