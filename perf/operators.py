"""The operators around the indexer: rotary positions of its queries and keys, and the attention that reads the
tokens it selects from a paged cache held in 8 bits (filling the cache, attending over it, weighing its tokens
by the attention they got, keeping the heaviest).

Each case is one call of one operator.  `run` computes it in elementary torch operations, in 32 bits (angles in
64), or, where `own` is true, through the package's entry points.
"""

import math

import torch

own = False

DEVICE = "cuda:0"
E4M3_MAX = 448.0
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


def listed():
    return [
        # One step of 16 sequences at far positions: the rotary part is the last 64 of 128 dimensions, adjacent pairs.
        dict(name="rotary_step", op="rotary", n0=1, n1=16, heads=64, dim=128, rot=64, start=64, layout="interleaved",
             dtype="bfloat16", max_pos=131072, yarn=False, grad=False),
        # A training pass over the index queries of the 4K workload, scaled for long contexts: forward and gradient.
        dict(name="rotary_train", op="rotary", n0=4096, n1=2, heads=64, dim=128, rot=64, start=0, layout="half",
             dtype="bfloat16", max_pos=32768, yarn=True, grad=True),
        # One new token for each of 32 sequences.
        dict(name="append_step", op="append", batch=32, new=1, kv_heads=8, dim=128, page=64, max_len=4096,
             dtype="bfloat16"),
        # Two prompts of 4096 tokens, into sequences that end inside a page.
        dict(name="append_prompt", op="append", batch=2, new=4096, kv_heads=8, dim=128, page=64, max_len=1000,
             dtype="bfloat16"),
        # A few drafted tokens checked at once over short contexts: odd group size, odd lengths, small pages.
        dict(name="attend_draft", op="attend", batch=3, queries=4, heads=15, kv_heads=5, dim=64, page=16, max_len=1025,
             dtype="float16", causal=True, ratio=1, topk=0),
        # One step of 16 sequences with up to 32K tokens in the cache.
        dict(name="attend_step", op="attend", batch=16, queries=1, heads=64, kv_heads=8, dim=128, page=64,
             max_len=32768, dtype="bfloat16", causal=False, ratio=1, topk=0),
        # Two prompts' second chunk of 4096 tokens, after 4096 in the cache.
        dict(name="attend_prompt", op="attend", batch=2, queries=4096, heads=32, kv_heads=4, dim=128, page=64,
             max_len=8192, dtype="bfloat16", causal=True, ratio=1, topk=0),
        # The tokens that the indexer selects: the 32K workload's compressed keys and topk, its last 4096 queries.
        dict(name="attend_selected", op="attend", batch=1, queries=4096, heads=64, kv_heads=1, dim=128, page=64,
             max_len=8192, dtype="bfloat16", causal=True, ratio=4, topk=2048),
        # What each cached token got from one step of 16 sequences.
        dict(name="weigh_step", op="weigh", batch=16, queries=1, heads=64, kv_heads=8, dim=128, page=64,
             max_len=32768, dtype="bfloat16", causal=False, ratio=1, topk=0),
        # What each cached token got from a prompt's chunk of 2048 queries.
        dict(name="weigh_prompt", op="weigh", batch=1, queries=2048, heads=32, kv_heads=4, dim=128, page=64,
             max_len=4096, dtype="bfloat16", causal=True, ratio=1, topk=0),
        # Short contexts cut to 256 tokens.
        dict(name="evict_short", op="evict", batch=4, kv_heads=8, dim=64, page=16, max_len=1000, keep=256, recent=64,
             sinks=4),
        # Contexts of up to 32K tokens cut to a quarter.
        dict(name="evict_long", op="evict", batch=8, kv_heads=8, dim=128, page=64, max_len=32768, keep=8192,
             recent=1024, sinks=4),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "attend", "weigh", "evict"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "rotary":
        dim = rng.choice([64, 80, 128, 128, 192])
        rot = rng.choice([32, 64, dim])
        heads = rng.choice([0, 1, 3, 8, 32, 64])
        n1 = _spread(rng, 1, 16)
        n0 = _spread(rng, 1, max(1, min(8192, (1 << 26) // (n1 * max(heads, 1) * dim))))
        return dict(op=op, n0=n0, n1=n1, heads=heads, dim=dim, rot=rot, start=rng.choice([0, dim - rot]),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bfloat16", "float16", "float32"]),
                    max_pos=_spread(rng, 1024, 1 << 20), yarn=rng.random() < 0.5, grad=rng.random() < 0.5)
    if op == "append":
        batch = _spread(rng, 1, 32)
        return dict(op=op, batch=batch, new=_spread(rng, 1, 8192 // batch), kv_heads=rng.choice([1, 2, 5, 8]), dim=dim,
                    page=page, max_len=_spread(rng, 1, 4096), dtype=dtype)
    if op == "evict":
        batch = _spread(rng, 1, 8)
        max_len = _spread(rng, 64, 32768)
        keep = _spread(rng, 16, max_len)
        recent = rng.randrange(0, keep // 2 + 1)
        return dict(op=op, batch=batch, kv_heads=rng.choice([1, 2, 5, 8]), dim=min(dim, 128), page=page,
                    max_len=max_len, keep=keep, recent=recent, sinks=rng.choice([0, 4, min(16, keep - recent)]))
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16]) if kv_heads > 1 else rng.choice([1, 8, 20, 64, 128])
    heads = kv_heads * group
    batch = _spread(rng, 1, 16)
    queries = rng.choice([1, 1, _spread(rng, 2, 8), _spread(rng, 9, 2048)])
    # keeps the products of a drawn case below those of the largest listed ones
    queries = max(1, min(queries, (1 << 18) // (batch * heads)))
    most = min(32768, (1 << 33) // (batch * heads * queries * dim))
    max_len = _spread(rng, 1 if rng.random() < 0.1 else min(200, most), most)
    topk = rng.choice([0, 0, 1]) if op == "attend" else 0
    if topk:
        topk = _spread(rng, min(64, max_len), min(2048, max_len, (1 << 26) // (batch * queries * kv_heads)))
    causal = queries > 1 or rng.random() < 0.3
    return dict(op=op, batch=batch, queries=queries, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                max_len=max_len, dtype=dtype, causal=causal, ratio=rng.choice([1, 1, 4]) if causal else 1, topk=topk)


# ------------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _lengths(case, g):
    """Tokens of each sequence: the longest first, the others between half of it and all; one of four or more is empty."""
    n, top = case["batch"], case["max_len"]
    lens = torch.randint((top + 1) // 2, top + 1, (n,), generator=g)
    lens[0] = top
    if n >= 4 and n % 2 == 1:
        lens[n // 2] = 0
    return lens.tolist()


def _table(counts, width, pages, g, first=0):
    """Pages of each sequence in a random order; -1 where it has none."""
    order = (torch.randperm(pages, generator=g) + first).tolist()
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [-1] * (width - c))
        at += c
    return _ints(rows)


def _inv_freq(rot, yarn):
    """Angle per position of each pair, radians; YaRN's blend for 16 times an original context of 4096 if asked."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if not yarn:
        return f, 1.0
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))   # noqa: E731
    low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
    keep = 1.0 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / 16.0 * (1.0 - keep) + f * keep, 0.1 * math.log(16.0) + 1.0


def _pool(pages, case, gpu):
    """A cache with every page filled: codes of values around one after scaling, scales a few octaves apart."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    pool = {}
    for x in ("k", "v"):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEVICE)
        step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
        for a in range(0, pages, step):
            part = torch.randn((min(step, pages - a),) + shape[1:], generator=gpu, device=DEVICE) * 60.0
            codes[a:a + step].view(torch.uint8).copy_(
                part.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
        pool[x] = codes
        pool[x + "_scale"] = (torch.rand(shape[:2], generator=gpu, device=DEVICE) * 2.0 - 1.0).exp2() / 60.0
    return pool


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed))
    gpu = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dtype = DTYPES[case.get("dtype", "bfloat16")]
    randn = lambda *shape: torch.randn(*shape, generator=gpu, device=DEVICE).to(dtype)   # noqa: E731
    s = dict(case)
    if case["op"] == "rotary":
        shape = (case["n0"], case["n1"]) + ((case["heads"],) if case["heads"] else ()) + (case["dim"],)
        s["x"] = randn(*shape).requires_grad_(case["grad"])
        s["dy"] = randn(*shape) if case["grad"] else None
        first = torch.randint(0, max(1, case["max_pos"] - case["n0"]), (1, case["n1"]), generator=g)
        s["positions"] = (first + torch.arange(case["n0"])[:, None]).to(torch.int32).to(DEVICE)
        f, s["scale"] = _inv_freq(case["rot"], case["yarn"])
        s["inv_freq"] = f.to(DEVICE)
        return s
    lens = _lengths(case, g)
    page, batch = case["page"], case["batch"]
    pages_of = lambda n: -(-n // page)   # noqa: E731
    if case["op"] == "append":
        new = [case["new"]] + torch.randint(0, case["new"] + 1, (batch,), generator=g).tolist()[1:]
        new = [case["new"]] * batch if case["new"] == 1 else new
        counts = [pages_of(a + b) for a, b in zip(lens, new)]
        width = pages_of(case["max_len"] + case["new"])
        s["pool"] = _pool(batch * width, case, gpu)
        s["table"] = _table(counts, width, batch * width, g)
        s["lens"], s["new_lens"] = _ints(lens), _ints(new)
        # keys and values as slices of one projection's output
        both = randn(batch, case["new"], 2 * case["kv_heads"], case["dim"])
        both = both * torch.rand(batch, case["new"], 1, 1, generator=gpu, device=DEVICE).mul_(4).exp2_().to(dtype)
        s["k"], s["v"] = both[:, :, :case["kv_heads"]], both[:, :, case["kv_heads"]:]
        return s
    counts = [pages_of(n) for n in lens]
    width = pages_of(case["max_len"])
    total = batch * width
    if case["op"] == "evict":
        kept = [pages_of(min(n, case["keep"])) for n in lens]
        new_width = pages_of(case["keep"])
        s["pool"] = _pool(total + batch * new_width, case, gpu)
        s["table"] = _table(counts, width, total, g)
        s["new_table"] = _table(kept, new_width, batch * new_width, g, first=total)
        s["lens"] = _ints(lens)
        # heavy tails, and many tokens with the same small weight
        w = torch.randn(batch, case["kv_heads"], width * page, generator=gpu, device=DEVICE).mul_(2).exp_()
        s["weights"] = torch.where(w < 0.3, torch.full_like(w, 0.125), w)
        return s
    s["pool"] = _pool(total, case, gpu)
    s["table"] = _table(counts, width, total, g)
    s["lens"] = _ints(lens)
    s["q"] = randn(batch, case["queries"], case["heads"], case["dim"])
    s["scale"] = case["dim"] ** -0.5
    s["q_start"] = s["q_lens"] = s["indices"] = None
    if case["causal"]:
        # the sequence ends with the last query: queries behind it are padding
        q_lens = [min(case["queries"], n * case["ratio"]) for n in lens]
        s["q_lens"] = _ints(q_lens)
        s["q_start"] = _ints([n * case["ratio"] - m for n, m in zip(lens, q_lens)])
    if case["topk"]:
        # as the top-k gives them: visible tokens in ascending order, -1 behind them
        queries, k = case["queries"], case["topk"]
        idx = torch.full((batch, queries, k), -1, dtype=torch.int32, device=DEVICE)
        t = torch.arange(queries, device=DEVICE)[:, None]
        for b, n in enumerate(lens):
            seen = torch.full((queries, 1), n, device=DEVICE)
            if case["causal"]:
                seen = torch.clamp((s["q_start"][b] + t + 1) // case["ratio"], max=n)
            score = torch.rand(queries, max(n, k), generator=gpu, device=DEVICE)
            score[torch.arange(max(n, k), device=DEVICE) >= seen] = -1.0
            best = torch.topk(score, k, dim=1)
            pick = torch.where(best.values < 0, n + k, best.indices).sort(dim=1).values
            idx[b] = torch.where(pick >= n + k, -1, pick)
        s["indices"] = idx
    if case["op"] == "weigh":
        s["lse"] = _attend(s)[1]
        s["weights"] = torch.zeros(batch, case["kv_heads"], width * page, device=DEVICE)
    return s


# ------------------------------------------------------------------ plain forms

def _rotate(x, positions, inv_freq, layout, start, scale, sign=1.0):
    rot = 2 * inv_freq.shape[0]
    angle = positions.double()[..., None] * inv_freq
    cos, sin = (angle.cos() * scale).float(), (angle.sin() * (scale * sign)).float()
    if x.dim() == 4:
        cos, sin = cos[:, :, None], sin[:, :, None]
    part = x[..., start:start + rot].float()
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :start], turned.to(x.dtype), x[..., start + rot:]], -1)


def _rotary(s):
    x = s["x"].detach()
    y = _rotate(x, s["positions"], s["inv_freq"], s["layout"], s["start"], s["scale"])
    if not s["grad"]:
        return y
    return y, _rotate(s["dy"], s["positions"], s["inv_freq"], s["layout"], s["start"], s["scale"], -1.0)


def _page_scale(top):
    """The smallest power of two, not below 2^-60, that brings `top` to at most 448."""
    m, e = torch.frexp(top / E4M3_MAX)          # top / 448 = m 2^e, 0.5 <= m < 1
    e = torch.where(top > 0, e - (m == 0.5).int(), -60).clamp(min=-60)
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _store(pool, name, page_ids, values, scale, write):
    """Writes values [n, kv_heads, page, dim] / scale [n, kv_heads] to the pages, where write [n, kv_heads, page]."""
    raw = pool[name].view(torch.uint8)
    codes = _codes(values, scale[..., None, None]).view(torch.uint8)
    raw[page_ids] = torch.where(write[..., None], codes, raw[page_ids])
    pool[name + "_scale"][page_ids] = scale


def _append(s):
    batch, new, heads, dim = s["k"].shape
    page, pool, lens = s["page"], s["pool"], s["lens"].long()
    # the pages that the new tokens fall on, of each sequence, and each slot's new token
    j = torch.arange((new + page - 1) // page + 1, device=lens.device)
    nth = lens[:, None] // page + j
    slot = nth[..., None] * page + torch.arange(page, device=lens.device)
    token = slot - lens[:, None, None]                                      # [batch, pages, page]
    fresh = (token >= 0) & (token < s["new_lens"].long()[:, None, None])
    live = fresh.any(-1)
    ids = torch.gather(s["table"].long(), 1, nth.clamp(max=s["table"].shape[1] - 1))[live]
    token, fresh, old = token.clamp(0, new - 1)[live], fresh[live], (token < 0)[live]
    b = torch.arange(batch, device=lens.device)[:, None].expand(live.shape)[live]
    for name in ("k", "v"):
        x = s[name][b[:, None], token].float().transpose(1, 2)               # [n, heads, page, dim]
        x = torch.where(fresh[:, None, :, None], x, torch.zeros((), device=x.device))
        before = pool[name + "_scale"][ids]
        need = _page_scale(x.abs().amax((-2, -1)))
        scale = torch.where(old.any(-1)[:, None], torch.maximum(before, need), need)
        kept = pool[name].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * before[..., None, None]
        x = torch.where(old[:, None, :, None], kept, x)
        _store(pool, name, ids, x, scale, (old | fresh)[:, None].expand(-1, heads, -1))
    return pool


def _tokens(pool, name, table, lens):
    """The cached values of each sequence, fp32 [batch, kv_heads, tokens, dim], zero behind its end."""
    batch, width = table.shape
    heads, page, dim = pool[name].shape[1:]
    at = table.long().clamp(min=0)
    x = pool[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    x = x * pool[name + "_scale"][at][..., None, None]
    x = x.transpose(1, 2).reshape(batch, heads, width * page, dim)
    behind = torch.arange(width * page, device=x.device) >= lens[:, None]
    return x.masked_fill(behind[:, None, :, None], 0.0)


def _visible(s, tokens):
    """How many of its sequence's tokens each query sees, [batch, queries]; none for a padded query."""
    batch, queries = s["q"].shape[:2]
    seen = s["lens"].long()[:, None].expand(batch, queries)
    if s["causal"]:
        t = torch.arange(queries, device=seen.device)
        seen = torch.minimum(seen, (s["q_start"].long()[:, None] + t + 1) // s["ratio"])
        seen = torch.where(t < s["q_lens"].long()[:, None], seen, torch.zeros_like(seen))
    return seen


def _softmax(x):
    """exp(x - lse) and lse over the last axis; 0 and -inf for rows that see nothing."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    return p / total.masked_fill(total == 0.0, 1.0), lse


def _scores(s, k):
    """Masked scores [batch, kv_heads, queries * group, tokens] of the whole sequences."""
    batch, queries, heads, dim = s["q"].shape
    q = s["q"].float().view(batch, queries, k.shape[1], -1, dim).transpose(1, 2)    # [b, kv, t, g, d]
    x = torch.matmul(q.reshape(batch, k.shape[1], -1, dim), k.transpose(-1, -2)).mul_(s["scale"])
    hidden = torch.arange(k.shape[2], device=k.device) >= _visible(s, k.shape[2])[..., None]
    x = x.view(batch, k.shape[1], queries, -1, k.shape[2])
    return x.masked_fill_(hidden[:, None, :, None], -math.inf)


def _attend(s):
    batch, queries, heads, dim = s["q"].shape
    k, v = (_tokens(s["pool"], n, s["table"], s["lens"]) for n in ("k", "v"))
    kv_heads = k.shape[1]
    if s["indices"] is None:
        p, lse = _softmax(_scores(s, k))                                            # [b, kv, t, g, tokens]
        out = torch.matmul(p.flatten(2, 3), v).view(batch, kv_heads, queries, -1, dim)
        out, lse = out.transpose(1, 2), lse.transpose(1, 2)
    else:
        at = s["indices"].long()
        hidden = (at < 0) | (at >= _visible(s, k.shape[2])[..., None])
        at = at.clamp(0, k.shape[2] - 1)
        b = torch.arange(batch, device=at.device)[:, None, None]
        rows = lambda x: x.transpose(1, 2)[b, at].permute(0, 1, 3, 2, 4).contiguous()   # noqa: E731
        x = torch.matmul(s["q"].float().view(batch, queries, kv_heads, -1, dim), rows(k).transpose(-1, -2))
        p, lse = _softmax((x * s["scale"]).masked_fill_(hidden[:, :, None, None], -math.inf))
        out = torch.matmul(p, rows(v))                                              # [b, t, kv, g, d]
    return out.reshape(batch, queries, heads, dim).to(s["q"].dtype), lse.reshape(batch, queries, heads).contiguous()


def _weigh(s):
    k = _tokens(s["pool"], "k", s["table"], s["lens"])
    batch, kv_heads, tokens, _ = k.shape
    x = _scores(s, k)
    lse = s["lse"].view(batch, s["queries"], kv_heads, -1).transpose(1, 2)[..., None]
    got = torch.exp(x - lse.masked_fill(lse == -math.inf, 0.0)).sum((2, 3))
    inside = torch.arange(tokens, device=k.device) < s["lens"][:, None]
    s["weights"].copy_(torch.where(inside[:, None], got, s["weights"]))
    return s["weights"]


def _evict(s):
    pool, page, keep, recent, sinks = s["pool"], s["page"], s["keep"], s["recent"], s["sinks"]
    w, lens = s["weights"], s["lens"].long()
    batch, heads, width = w.shape
    at = torch.arange(width, device=w.device)
    # first and last tokens before all others, then by weight, then by index
    must = (at < sinks) | (at >= (lens - recent)[:, None])                             # [batch, width]
    rank = torch.where(must[:, None], torch.full_like(w, math.inf), w)
    rank = rank.masked_fill((at >= lens[:, None])[:, None], -math.inf)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    first = torch.nn.functional.pad(first, (0, max(0, keep - width)), value=width)
    count = lens.clamp(max=keep)
    slot = torch.arange(keep, device=w.device)
    inside = (slot < count[:, None])[:, None].expand(-1, heads, -1)
    kept = torch.sort(torch.where(inside, first, torch.full_like(first, width)), dim=-1).values
    src = torch.where(inside, kept, torch.zeros_like(kept))
    new_w = torch.where(inside, torch.gather(w, 2, src), torch.zeros((), device=w.device))
    # the kept tokens, page by page of the new table
    pages = s["new_table"].shape[1]
    pad = lambda x, v: torch.nn.functional.pad(x, (0, pages * page - keep), value=v)   # noqa: E731
    src, full = pad(src, 0), pad(inside, False).view(batch, heads, pages, page).transpose(1, 2)
    old = torch.gather(s["table"].long()[:, None].expand(-1, heads, -1), 2, src // page).clamp(min=0)
    h = torch.arange(heads, device=w.device)[:, None]
    live = full.any(-1).any(-1)
    ids = s["new_table"].long()[live]
    for name in ("k", "v"):
        x = pool[name].view(torch.uint8)[old, h, src % page].view(torch.float8_e4m3fn).float()
        x = x * pool[name + "_scale"][old, h][..., None]
        x = x.view(batch, heads, pages, page, -1).transpose(1, 2)[live]
        x = torch.where(full[live][..., None], x, torch.zeros((), device=w.device))
        _store(pool, name, ids, x, _page_scale(x.abs().amax((-2, -1))), full[live])
    return dict(pool, new_lens=count.to(torch.int32), kept=torch.where(inside, kept, -torch.ones_like(kept)).to(torch.int32),
                weights=new_w)


def run(state):
    s = state
    if not own:
        return {"rotary": _rotary, "append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[s["op"]](s)
    import sparse_attention_lightning_bf16_amd as lx
    if s["op"] == "rotary":
        y = lx.rotary(s["x"], s["positions"], s["inv_freq"], layout=s["layout"], start=s["start"], scale=s["scale"])
        if not s["grad"]:
            return y
        return y.detach(), torch.autograd.grad(y, s["x"], s["dy"])[0]
    pool = s["pool"]
    cache = lx.KV8Cache(pool["k"], pool["v"], pool["k_scale"], pool["v_scale"])
    if s["op"] == "append":
        lx.kv8_append(cache, s["k"], s["v"], s["table"], s["lens"], new_lens=s["new_lens"])
        return pool
    if s["op"] == "attend":
        return lx.kv8_attention(s["q"], cache, s["table"], s["lens"], q_start=s["q_start"], q_lens=s["q_lens"],
                                compress_ratio=s["ratio"], scale=s["scale"], topk_indices=s["indices"])
    if s["op"] == "weigh":
        return lx.kv8_token_weights(s["q"], cache, s["table"], s["lens"], s["lse"], q_start=s["q_start"],
                                    q_lens=s["q_lens"], compress_ratio=s["ratio"], scale=s["scale"],
                                    out=s["weights"])
    new_lens, kept, weights = lx.kv8_evict(cache, s["table"], s["lens"], s["weights"], s["new_table"], s["keep"],
                                           recent=s["recent"], sinks=s["sinks"])
    return dict(pool, new_lens=new_lens, kept=kept, weights=weights)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rotary(s):
    def turn(x, sign):
        x = x.detach().double()
        y = x.clone()
        half = s["rot"] // 2
        for i in range(half):
            a, b = (i, i + half) if s["layout"] == "half" else (2 * i, 2 * i + 1)
            a, b = a + s["start"], b + s["start"]
            angle = s["positions"].double() * s["inv_freq"][i]
            c, d = angle.cos() * s["scale"], sign * angle.sin() * s["scale"]
            if x.dim() == 4:
                c, d = c[..., None], d[..., None]
            y[..., a] = x[..., a] * c - x[..., b] * d
            y[..., b] = x[..., b] * c + x[..., a] * d
        return y
    return (turn(s["x"], 1.0), turn(s["dy"], -1.0)) if s["grad"] else turn(s["x"], 1.0)


def _exact_cache(s):
    """Each sequence's cached keys and values in 64 bits, a list of [kv_heads, tokens, dim] pairs."""
    found = []
    for b, n in enumerate(s["lens"].tolist()):
        pair = []
        for name in ("k", "v"):
            ids = s["table"][b, :-(-n // s["page"])].long()
            x = s["pool"][name].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            x = x * s["pool"][name + "_scale"][ids].double()[:, :, None, None]
            pair.append(x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n])
        found.append(pair)
    return found


def _exact_attention(s):
    batch, queries, heads, dim = s["q"].shape
    group = heads // s["kv_heads"]
    out = torch.zeros(batch, queries, heads, dim, dtype=torch.float64, device=DEVICE)
    lse = torch.full((batch, queries, heads), -math.inf, dtype=torch.float64, device=DEVICE)
    weights = None
    if s["op"] == "weigh":
        weights = s["weights"].double()
    for b, (k, v) in enumerate(_exact_cache(s)):
        n = k.shape[1]
        if n == 0:
            continue
        t = torch.arange(queries, device=DEVICE)
        seen = torch.full((queries,), n, device=DEVICE)
        if s["causal"]:
            seen = ((int(s["q_start"][b]) + t + 1) // s["ratio"]).clamp(max=n)
            seen[t >= int(s["q_lens"][b])] = 0
        count = (torch.arange(n, device=DEVICE) < seen[:, None]).double()
        if s["indices"] is not None:
            listed_at = s["indices"][b].long()
            times = torch.zeros(queries, n + 1, dtype=torch.float64, device=DEVICE)
            times.scatter_add_(1, torch.where((listed_at < 0) | (listed_at >= n), n, listed_at),
                               torch.ones_like(listed_at, dtype=torch.float64))
            count = count * times[:, :n]
        for h in range(heads):
            x = torch.mm(s["q"][b, :, h].double(), k[h // group].t().contiguous()) * s["scale"]
            x = x.masked_fill(count == 0, -math.inf)
            if weights is not None:
                if h % group == 0:
                    weights[b, h // group, :n] = 0.0
                ref = s["lse"][b, :, h].double()
                weights[b, h // group, :n] += torch.exp(x - ref.masked_fill(ref == -math.inf, 0.0)[:, None]).sum(0)
                continue
            top = x.amax(1, keepdim=True).nan_to_num(neginf=0.0)
            p = torch.exp(x - top) * count
            total = p.sum(1, keepdim=True)
            out[b, :, h] = torch.mm(p, v[h // group]) / total.masked_fill(total == 0, 1.0)
            lse[b, :, h] = (top + total.log())[:, 0]
    return (out, lse) if weights is None else weights


def _exact_scale(top):
    return 2.0 ** max(-60, math.ceil(math.log2(top / E4M3_MAX))) if top > 0 else 2.0 ** -60


def _exact_append(s):
    """Quotients before their rounding to 8 bits; codes that were there stay unless their page's scale grew."""
    got = {x: s["pool"][x].double() for x in s["pool"]}
    page = s["page"]
    for b, (n, new) in enumerate(zip(s["lens"].tolist(), s["new_lens"].tolist())):
        for i in range(n // page, -(-(n + new) // page) if new else 0):
            at = int(s["table"][b, i])
            lo, hi = max(n, i * page), min(n + new, (i + 1) * page)
            for name in ("k", "v"):
                x = s[name][b, lo - n:hi - n].double().transpose(0, 1)
                scales = torch.tensor([_exact_scale(t) for t in x.abs().amax((1, 2)).tolist()], dtype=torch.float64,
                                      device=DEVICE)
                if lo > i * page:
                    scales = torch.maximum(scales, got[name + "_scale"][at])
                    got[name][at, :, :lo - i * page] *= (got[name + "_scale"][at] / scales)[:, None, None]
                got[name][at, :, lo - i * page:hi - i * page] = x / scales[:, None, None]
                got[name + "_scale"][at] = scales
    return got


def _exact_evict(s):
    """Quotients before their rounding to 8 bits, and the kept tokens' weights; whole numbers have no such value."""
    got = {x: s["pool"][x].double() for x in s["pool"]}
    cache = _exact_cache(s)
    page, keep = s["page"], s["keep"]
    got["weights"] = torch.zeros(s["batch"], s["kv_heads"], keep, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(s["lens"].tolist()):
        count = min(n, keep)
        for h in range(s["kv_heads"]):
            w = s["weights"][b, h, :n].double().cpu().tolist()
            ends = set(range(min(s["sinks"], n))) | set(range(max(0, n - s["recent"]), n))
            rest = sorted((i for i in range(n) if i not in ends), key=lambda i: (-w[i], i))
            chosen = list(range(n)) if n <= keep else sorted(list(ends) + rest[:keep - len(ends)])
            pick = torch.tensor(chosen, dtype=torch.int64, device=DEVICE)
            got["weights"][b, h, :count] = s["weights"][b, h, :n].double()[pick]
            for x, name in zip(cache[b], ("k", "v")):
                rows = x[h, pick]
                spare = -count % page
                tops = torch.nn.functional.pad(rows, (0, 0, 0, spare)).view(-1, page * s["dim"]).abs().amax(1)
                ids = s["new_table"][b, :len(tops)].long()
                scales = torch.tensor([_exact_scale(t) for t in tops.tolist()], dtype=torch.float64, device=DEVICE)
                of_row = scales.repeat_interleave(page)[:count]
                place = torch.arange(count, device=DEVICE)
                got[name][ids[place // page], h, place % page] = rows / of_row[:, None]
                got[name + "_scale"][ids, h] = scales
    return dict(got, new_lens=None, kept=None)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "attend": _exact_attention, "weigh": _exact_attention,
            "evict": _exact_evict}[s["op"]](s)


# ------------------------------------------------------------------ the work

def work(case):
    """Bytes and operations of a pass; lengths as on average over the seeds."""
    op = case["op"]
    if op == "rotary":
        n = case["n0"] * case["n1"] * max(1, case["heads"]) * case["dim"]
        size = 4 if case["dtype"] == "float32" else 2
        passes = 2 if case["grad"] else 1
        return {"bytes": passes * 2 * n * size, "flops": passes * 3 * n}
    rows = case["kv_heads"] * case["dim"]
    mean = (case["max_len"] * (1 + 0.75 * (case["batch"] - 1))) / case["batch"]
    if op == "append":
        tokens = case["batch"] * case["new"] * (1.0 if case["new"] == 1 else (1 + 0.5 * (case["batch"] - 1)) / case["batch"])
        return {"bytes": tokens * rows * 2 * (2 + 1), "flops": tokens * rows * 2 * 2}
    if op == "evict":
        kept = case["batch"] * min(mean, case["keep"])
        return {"bytes": 4 * case["batch"] * case["kv_heads"] * mean + kept * rows * 2 * 2, "flops": kept * rows * 2 * 2}
    seen = mean
    if case["causal"]:
        seen = max(1.0, mean - (case["queries"] - 1) / (2 * case["ratio"]))
    pairs = case["batch"] * case["queries"] * case["heads"] * (min(seen, case["topk"]) if case["topk"] else seen)
    q_bytes = 2 * case["batch"] * case["queries"] * case["heads"] * case["dim"]
    cached = case["batch"] * mean * rows
    if case["topk"]:
        cached = min(cached, case["batch"] * case["queries"] * case["topk"] * rows)
    if op == "weigh":
        return {"bytes": cached + q_bytes + 4 * case["batch"] * mean * case["kv_heads"], "flops": 2 * pairs * case["dim"]}
    index = 4 * case["batch"] * case["queries"] * case["topk"]
    return {"bytes": 2 * cached + 2 * q_bytes + index, "flops": 4 * pairs * case["dim"]}
