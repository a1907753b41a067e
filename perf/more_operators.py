"""Workloads of the second set of serving operators: queries and keys normed
per head and rotated in one pass (into a paged cache, or dense before the
prompt's attention; positions of one or several axes), attention of a batch
whose sequences share a long prefix, the attention weight that a cache's
tokens gather, and eviction of the lightest tokens.

Sizes come from the library's own configurations (32 heads of 128, 40 heads
of 96, 2 heads of 64, grouped-query attention of 32 over 8 heads, contexts of
2K to 32K, pages of 16 to 128) or are generic serving sizes.
"""
import math
import random

import torch

own = False

TWO_PI = 2.0 * math.pi
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _case(op, name, **fields):
    c = dict(op=op, **fields)
    return dict(c, name=name) if name else c


def _append(name, batch, heads, kv_heads, head_dim, page, ctx, new, ragged, rotary, pairs, axes, with_q, per_head, weight):
    return _case("append", name, batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, ctx=ctx, new=new,
                 ragged=ragged, rotary=rotary, pairs=pairs, axes=axes, with_q=with_q, per_head=per_head, weight=weight)


def _rotate_case(name, batch, heads, kv_heads, head_dim, new, rotary, pairs, axes, per_head, weight):
    return _case("rotate", name, batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, new=new, rotary=rotary,
                 pairs=pairs, axes=axes, per_head=per_head, weight=weight)


def _prefix(name, groups, members, heads, kv_heads, head_dim, page, prefix, suffix, new, branch, ragged):
    return _case("prefix", name, groups=groups, members=members, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                 prefix=prefix, suffix=suffix, new=new, branch=branch, ragged=ragged)


def _weights(name, batch, heads, kv_heads, head_dim, page, ctx, new, ragged):
    return _case("weights", name, batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, ctx=ctx, new=new,
                 ragged=ragged)


def _evict(name, batch, kv_heads, head_dim, page, ctx, budget, recent, sink, ragged):
    return _case("evict", name, batch=batch, kv_heads=kv_heads, head_dim=head_dim, page=page, ctx=ctx, budget=budget,
                 recent=recent, sink=sink, ragged=ragged)


def listed():
    return [
        # a prompt of 32K enters the cache: queries and keys normed and rotated on the way
        _append("append_prompt_32k", 1, 32, 8, 128, 128, 0, 32768, False, 128, False, 1, True, False, "bf16"),
        # one token of each of 64 users
        _append("append_token_b64", 64, 32, 8, 128, 64, 8192, 1, True, 128, False, 1, True, False, "bf16"),
        # the patches of two images between text: three axes, neighbouring pairs, every head with weights of its own
        _append("append_image_d96", 2, 40, 40, 96, 16, 517, 4099, True, 96, True, 3, True, True, "f32"),
        # a prompt's queries and keys before its attention, dense
        _rotate_case("rotate_prompt_16k", 1, 32, 32, 128, 16384, 128, False, 1, False, "bf16"),
        # a short one with small heads, half of each head rotated by three axes
        _rotate_case("rotate_short_d64", 3, 8, 2, 64, 77, 32, False, 3, False, "f32"),
        # next tokens of 64 users behind one long instruction text
        _prefix("prefix_token_b64_32k", 1, 64, 32, 8, 128, 64, 32768, 1024, 1, 1, True),
        # a few samples of one short prompt, small heads, small pages
        _prefix("prefix_short_d64", 1, 5, 8, 2, 64, 16, 333, 77, 3, 2, True),
        # drafted trees in three groups of users, each group with its own text
        _prefix("prefix_tree_groups_d96", 3, 8, 40, 8, 96, 32, 8192, 700, 5, 2, True),
        # the last 32 tokens of a prompt of 32K weigh what stands before them
        _weights("weights_window_32k", 1, 32, 8, 128, 128, 32736, 32, False),
        # next tokens of 32 users
        _weights("weights_token_b32_8k", 32, 32, 8, 128, 64, 8192, 1, True),
        # a prompt of 32K is cut down to 2K tokens a head
        _evict("evict_prompt_32k", 1, 8, 128, 64, 32768, 2048, 32, 4, False),
        # a server's caches fall to half of 8K
        _evict("evict_b16_8k", 16, 8, 128, 32, 8192, 4096, 128, 4, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (32, 32, 128), (40, 40, 96), (8, 2, 64), (32, 4, 64), (40, 8, 96),
                                       (16, 1, 128), (2, 2, 64)])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    op = rng.choice(["append", "rotate", "prefix", "prefix", "weights", "evict"])
    batch = _log(rng, 1, 64)
    axes, pairs = rng.choice([1, 1, 2, 3]), rng.random() < 0.5
    per_head, weight = rng.random() < 0.3, rng.choice(["bf16", "f32"])
    rotary = rng.choice([dim, dim, dim // 2, 32])
    if op in ("append", "rotate"):
        new, ctx = _log(rng, 1, 32768), rng.choice([0, _log(rng, 1, 32768)])
        with_q = rng.random() < 0.7
        while batch * new * (2 * heads + 4 * kv_heads) * dim * 2 > 8e8 or batch * (ctx + new) * kv_heads > 2 ** 21:
            if batch > 1 and rng.random() < 0.5:
                batch = (batch + 1) // 2
            else:
                new, ctx = max(1, new // 2), ctx // 2
        if op == "rotate":
            return _rotate_case(None, batch, heads, kv_heads, dim, new, rotary, pairs, axes, per_head, weight)
        return _append(None, batch, heads, kv_heads, dim, page, ctx, new, ragged, rotary, pairs, axes, with_q, per_head, weight)
    if op == "prefix":
        groups = rng.choice([1, 1, 2, 3])
        members, prefix, suffix = _log(rng, 1, 128), _log(rng, 1, 65536), _log(rng, 1, 4096)
        new, branch = _log(rng, 1, 64), rng.choice([1, 2, 3])
        case = lambda: _prefix(None, groups, members, heads, kv_heads, dim, page, prefix, suffix, new, branch, ragged)  # noqa: E731
        while (work(case())["bytes"] > 4e8 or work(case())["flops"] > 6e10
               or groups * members * heads * new * (prefix + suffix) > 2 ** 27):
            if members > 1 and rng.random() < 0.5:
                members = (members + 1) // 2
            else:
                prefix, suffix = max(1, prefix // 2), max(1, suffix - suffix // 4)
                new = max(1, new - new // 4)
        return case()
    if op == "weights":
        new, ctx = _log(rng, 1, 128), _log(rng, 1, 131072)
        while batch * (ctx + new) * kv_heads * dim * 2 > 4e8 or batch * heads * new * ctx > 2 ** 27:
            if batch > 1 and rng.random() < 0.5:
                batch = (batch + 1) // 2
            else:
                ctx, new = max(1, ctx // 2), max(1, new - new // 8)
        return _weights(None, batch, heads, kv_heads, dim, page, ctx, new, ragged)
    ctx = _log(rng, 1, 131072)
    while batch * ctx * kv_heads * dim * 8 > 8e8:
        batch, ctx = (batch + 1) // 2, max(1, ctx - ctx // 3)
    budget = max(1, min(ctx, int(ctx * rng.uniform(0.05, 1.1))))
    recent = rng.randint(0, budget // 2)
    sink = rng.randint(0, min(8, budget - recent))
    return _evict(None, batch, kv_heads, dim, page, ctx, budget, recent, sink, ragged)


def _lengths(case):
    """Committed tokens and new tokens of each sequence."""
    if case["op"] == "prefix":
        sizes, prefixes = _groups(case)
        lengths = []
        for m, x in zip(sizes, prefixes):
            for i in range(m):
                s = case["suffix"]
                lengths.append(x + (s if not case["ragged"] else max(0, s - (s * ((5 * i) % 8)) // 9 - i % 3)))
        new = case["new"]
        return lengths, [new if not case["ragged"] else max(1, new - (new * (i % 4)) // 4) for i in range(len(lengths))]
    b, ctx, new = case["batch"], case["ctx"], case.get("new", 0)
    if not case["ragged"]:
        return [ctx] * b, [new] * b
    lengths = [max(0, ctx - (ctx * ((5 * i) % 8)) // 9 - i % 3) for i in range(b)]
    return lengths, [max(1, new - (new * (i % 4)) // 4) for i in range(b)]


def _groups(case):
    """Sequences and shared tokens of each group."""
    m, p = case["members"], case["prefix"]
    if not case["ragged"]:
        return [m] * case["groups"], [p] * case["groups"]
    return ([max(1, m - (m * (g % 3)) // 4) for g in range(case["groups"])],
            [max(1, p - (p * (g % 3)) // 5 - g % 2) for g in range(case["groups"])])


def _depths(case):
    """Depth of each drafted token: token i hangs below token (i - 1) // branch, the first below the context."""
    depth = [0] * case["new"]
    for i in range(1, case["new"]):
        depth[i] = depth[(i - 1) // case["branch"]] + 1
    return depth


def work(case):
    op, hk, d = case["op"], case["kv_heads"], case["head_dim"]
    if op == "rotate":
        rows = case["batch"] * case["new"] * (case["heads"] + hk)
        return {"bytes": rows * d * 4, "flops": rows * (4 * d + 3 * case["rotary"])}
    lengths, news = _lengths(case)
    if op == "append":
        tokens, q = sum(news), case["batch"] * case["new"] * case["heads"] if case["with_q"] else 0
        return {"bytes": tokens * hk * d * 8 + q * d * 4, "flops": (tokens * hk + q) * (4 * d + 3 * case["rotary"])}
    if op == "evict":
        kept = [min(x, case["budget"]) for x in lengths]
        moved = sum(kept)
        return {"bytes": hk * (moved * d * 8 + sum(lengths) * 4 + moved * 4), "flops": 0}
    h, n = case["heads"], case["new"]
    if op == "weights":
        keys = sum(x + y for x, y in zip(lengths, news))
        pairs = sum(x * y + y * (y + 1) // 2 for x, y in zip(lengths, news))
        return {"bytes": keys * hk * (d * 2 + 8) + sum(news) * h * (d * 2 + 4), "flops": 2 * d * h * pairs}
    depth = _depths(case)
    sizes, prefixes = _groups(case)
    keys = sum(lengths) + sum(news) - sum((m - 1) * x for m, x in zip(sizes, prefixes))
    pairs = sum(x * y + sum(depth[:y]) + y for x, y in zip(lengths, news))
    rows = len(lengths) * n * h
    return {"bytes": keys * hk * d * 4 + sum(news) * h * d * 2 + rows * (d * 2 + 4), "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ inputs

def _mask_words(case):
    """[n, ceil(n / 32)] int32: bit j % 32 of word j // 32 of row i: drafted token i sees drafted token j."""
    n = case["new"]
    rows = []
    for i in range(n):
        rows.append((1 << i) | (rows[(i - 1) // case["branch"]] if i else 0))
    words = [[(r >> (32 * w)) & 0xffffffff for w in range((n + 31) // 32)] for r in rows]
    return torch.tensor([[x - (1 << 32) if x >> 31 else x for x in r] for r in words], dtype=torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, hk, d = case["op"], case["kv_heads"], case["head_dim"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(torch.bfloat16)

    st = dict(case=case)
    if op in ("append", "rotate"):
        _prepare_rotation(st, normal, g, dev)
    if op == "rotate":
        return st
    page = case["page"]
    lengths, news = _lengths(case)
    b = len(lengths)
    used = [(x + y + page - 1) // page for x, y in zip(lengths, news)]
    max_pages = max(max(used), 1) + 1
    # whole pages of a group's prefix lie in the pool once
    shared, leader = [0] * b, list(range(b))
    if op == "prefix":
        sizes, prefixes = _groups(case)
        at = 0
        for m, x in zip(sizes, prefixes):
            for i in range(at, at + m):
                shared[i], leader[i] = (0, i) if i == at else (x // page, at)
            at += m
    kept = [(min(x, case["budget"]) + page - 1) // page for x in lengths] if op == "evict" else [0] * b
    n_pages = sum(used) - sum(shared) + sum(kept) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    table = [[-1] * max_pages for _ in range(b)]
    for i in range(b):
        table[i][:shared[i]] = table[leader[i]][:shared[i]]
        for c in range(shared[i], used[i]):
            table[i][c] = order.pop()
    st.update(k_pages=normal(n_pages, hk, page, d), v_pages=normal(n_pages, hk, page, d),
              table=torch.tensor(table, dtype=torch.int32, device=dev),
              lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
              new_len=torch.tensor(news, dtype=torch.int32, device=dev) if case["ragged"] and op != "evict" else None,
              news=torch.tensor(news, dtype=torch.int32, device=dev))
    if op == "append":
        i = torch.arange(case["new"], device=dev)
        st["token"] = torch.nonzero(i[None] < torch.tensor(news, device=dev)[:, None], as_tuple=True)
        if st["positions"] is not None:
            st["positions"] = (st["positions"] + st["lengths"][None, :, None]).contiguous()
    elif op == "prefix":
        sizes, prefixes = _groups(case)
        # queries of a few units' length: some keys stand out
        st["q"] = normal(b, case["heads"], case["new"], d, scale=1.5)
        st["mask"] = None if case["branch"] == 1 else _mask_words(case).to(dev)[None].expand(b, -1, -1).contiguous()
        starts = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        st["prefix"] = torch.tensor(prefixes, dtype=torch.int32, device=dev)
        for m, x, s in zip(sizes, prefixes, starts):
            if x % page:  # the page in which the prefix ends: each sequence has its own
                first, rest = table[s][x // page], [table[i][x // page] for i in range(s + 1, s + m)]
                for pool in (st["k_pages"], st["v_pages"]):
                    pool[rest, :, :x % page] = pool[first, :, :x % page]
    elif op == "weights":
        st["q"] = normal(b, case["heads"], case["new"], d, scale=1.5)
        width = max(lengths) + max(news) + 5
        # what earlier tokens left: few tokens hold most of it
        st["weights"] = torch.exp(3.0 * torch.randn((b, hk, width), generator=g, device=dev) - 4.0)
        lse = []
        for i in range(b):  # as the attention of these tokens returned it
            p, _ = _scores(st, i)
            lse.append(torch.logsumexp(p, -1))
        st["lse"] = torch.stack(lse).contiguous()
    else:
        new_pages = max(max(kept), 1) + 1
        st["to"] = torch.tensor([[order.pop() for _ in range(k)] + [-1] * (new_pages - k) for k in kept], dtype=torch.int32, device=dev)
        width = max(lengths) + 5
        # few tokens hold most of the weight, and some hold none at all
        w = torch.exp(3.0 * torch.randn((b, hk, width), generator=g, device=dev) - 4.0)
        none = torch.rand((b, hk, width), generator=g, device=dev) < 0.1
        st["weights"] = torch.where(none, 0.0, w)
    return st


def _prepare_rotation(st, normal, g, dev):
    case = st["case"]
    b, h, hk, d, n, r = (case[x] for x in ("batch", "heads", "kv_heads", "head_dim", "new", "rotary"))
    # one projection's output holds queries, keys and values of a token side by side
    qkv = normal(b, n, h + 2 * hk, d).transpose(1, 2)
    st["q"] = qkv[:, :h] if case.get("with_q", True) else None
    st["k"], st["v"] = qkv[:, h:h + hk], qkv[:, h + hk:]
    kind = torch.float32 if case["weight"] == "f32" else torch.bfloat16

    def weights(heads):
        shape = (heads, d) if case["per_head"] else (d,)
        return (1.0 + 0.2 * torch.randn(shape, generator=g, device=dev)).to(kind)

    st["q_norm"], st["k_norm"] = weights(h) if st["q"] is not None else None, weights(hk)
    inv_freq = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    st["inv_freq"] = torch.tensor(inv_freq, dtype=torch.float64, device=dev)
    # turns per position in units of 2^-64, as signed 64-bit whole numbers
    steps = [int(round(f / TWO_PI * 2.0 ** 64)) for f in inv_freq]
    st["steps"] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in steps], dtype=torch.int64, device=dev)
    st["axes"] = st["positions"] = None
    a = case["axes"]
    if a > 1:
        # time, rows and columns of an image (rows and columns alone with two axes), a share of the pairs each
        st["axes"] = torch.tensor([i * a // (r // 2) for i in range(r // 2)], dtype=torch.int32, device=dev)
        i, wide = torch.arange(n, device=dev), max(1, math.isqrt(n))
        at = [torch.zeros_like(i), i // wide, i % wide][3 - a:]
        st["positions"] = torch.stack(at)[:, None].expand(a, b, n).to(torch.int32).contiguous()


def _scores(st, i):
    """Scores of sequence i's new tokens in 32 bits, [heads, n, keys], and which are seen (the rest is -inf)."""
    case = st["case"]
    h, hk, d, n = (case[x] for x in ("heads", "kv_heads", "head_dim", "new"))
    length, new = int(st["lengths"][i]), int(st["news"][i])
    page = case["page"]
    pages = st["table"][i, :(length + new + page - 1) // page].long()
    k = st["k_pages"][pages].transpose(0, 1).reshape(hk, -1, d)[:, :length + new].float()
    s = (st["q"][i].float().reshape(hk, -1, d) @ k.transpose(1, 2)).reshape(h, n, -1) / math.sqrt(d)
    key, row = torch.arange(length + new, device="cuda"), torch.arange(n, device="cuda")[:, None]
    seen = (row < new) & (key - length <= row)
    return s.masked_fill(~seen, -math.inf), seen


# -------------------------------------------------------------- plain forms

def _slots(st, batch, token):
    """Page and row of token `token` behind the committed ones of sequence `batch`."""
    page = st["k_pages"].shape[2]
    pos = st["lengths"].long()[batch] + token
    return st["table"].long()[batch, pos // page], pos % page


def _norm_rotate(x, weight, angle, pairs):
    """x [b, heads, n, d], angle [b, n, r / 2] in 64 bits; in 32 bits."""
    x = x.float()
    w = weight.float()
    w = w[:, None] if w.dim() == 2 else w
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = angle.shape[-1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if pairs:
        a, b = rot[..., 0::2], rot[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2), rest], dim=-1)
    a, b = rot[..., :half], rot[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], dim=-1)


def _angles(st):
    """[b, n, r / 2] in 64 bits."""
    case = st["case"]
    b, n = case["batch"], case["new"]
    if st["positions"] is None:
        at = torch.arange(n, device="cuda").expand(b, n)
        if "lengths" in st:
            at = at + st["lengths"][:, None]
        return at.double()[..., None] * st["inv_freq"]
    return st["positions"].double()[st["axes"].long()].permute(1, 2, 0) * st["inv_freq"]


def _plain_append(st):
    case = st["case"]
    angle = _angles(st)
    b, i = st["token"]
    page, row = _slots(st, b, i)
    k = _norm_rotate(st["k"], st["k_norm"], angle, case["pairs"]).to(torch.bfloat16)
    st["k_pages"][page, :, row] = k[b, :, i]
    st["v_pages"][page, :, row] = st["v"][b, :, i]
    out = {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if st["q"] is not None:
        out["q"] = _norm_rotate(st["q"], st["q_norm"], angle, case["pairs"]).to(torch.bfloat16)
    return out


def _plain_rotate(st):
    angle, pairs = _angles(st), st["case"]["pairs"]
    return {"q": _norm_rotate(st["q"], st["q_norm"], angle, pairs).to(torch.bfloat16),
            "k": _norm_rotate(st["k"], st["k_norm"], angle, pairs).to(torch.bfloat16)}


def _plain_prefix(st):
    """Group by group: the shared keys once against all of the group's rows, each sequence's own ones after them."""
    case = st["case"]
    h, hk, d, n, page = (case[x] for x in ("heads", "kv_heads", "head_dim", "new", "page"))
    sizes, prefixes = _groups(case)
    table = st["table"].long()
    outs, lses, at = [], [], 0
    for m, x in zip(sizes, prefixes):
        whole = x // page
        mine = slice(at, at + m)
        # [hk, tokens, d], shared; [m, hk, tokens, d], own
        def pool(name):
            p = st[name]
            return (p[table[at, :whole]].transpose(0, 1).reshape(hk, whole * page, d).float(),
                    p[table[mine, whole:]].transpose(1, 2).reshape(m, hk, -1, d).float())
        k, k_own = pool("k_pages")
        v, v_own = pool("v_pages")
        each = h // hk * n  # rows of a sequence and key head
        q = st["q"][mine].float().reshape(m, hk, each, d)
        rows = q.transpose(0, 1).reshape(hk, m * each, d)
        s = (rows @ k.transpose(1, 2)).reshape(hk, m, each, whole * page).transpose(0, 1) / math.sqrt(d)
        s_own = q @ k_own.transpose(2, 3) / math.sqrt(d)  # [m, hk, group * n, keys]
        key = whole * page + torch.arange(k_own.shape[2], device="cuda")
        length, news = st["lengths"].long()[mine, None, None], st["news"].long()[mine, None, None]
        j = key[None, None] - length
        row = torch.arange(n, device="cuda")[None, :, None]
        if st["mask"] is None:
            sees = j <= row
        else:
            to = j.clamp(0, n - 1).expand(m, n, -1)
            sees = (torch.gather(st["mask"][mine], 2, to // 32) >> (to % 32).int()) & 1 == 1
        live = row < news
        seen = live & ((j < 0) | ((j < news) & sees))  # [m, n, keys]
        s = s.reshape(m, h, n, whole * page).masked_fill(~live[:, None], -math.inf)
        s_own = s_own.reshape(m, h, n, -1).masked_fill(~seen[:, None], -math.inf)
        both = torch.cat([s, s_own], -1)
        top = both.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), 0.0, top)
        p = torch.exp(both - top)
        total = p.sum(-1, keepdim=True)
        p, p_own = p[..., :s.shape[-1]], p[..., s.shape[-1]:]
        p = p.reshape(m, hk, each, whole * page).transpose(0, 1).reshape(hk, m * each, whole * page)
        o = (p @ v).reshape(hk, m, each, d).transpose(0, 1) + p_own.reshape(m, hk, each, p_own.shape[-1]) @ v_own
        outs.append(torch.where(total > 0, o.reshape(m, h, n, d) / total, 0.0))
        lses.append((torch.log(total) + top)[..., 0])
        at += m
    return {"out": torch.cat(outs).to(torch.bfloat16), "lse": torch.cat(lses)}


def _plain_weights(st):
    case = st["case"]
    b, h, hk, d, n = (case[x] for x in ("batch", "heads", "kv_heads", "head_dim", "new"))
    k = st["k_pages"][st["table"].long()].transpose(1, 2).reshape(b, hk, -1, d).float()
    width = st["weights"].shape[2]
    most = min(k.shape[2], width)
    s = (st["q"].float().reshape(b, hk, -1, d) @ k[:, :, :most].transpose(2, 3)).reshape(b, h, n, -1) / math.sqrt(d)
    length, news = st["lengths"].long()[:, None, None], st["news"].long()[:, None, None]
    j = torch.arange(most, device="cuda")[None, None] - length
    row = torch.arange(n, device="cuda")[None, :, None]
    seen = (row < news) & (j <= row) & (j < news)
    p = torch.exp((s - st["lse"][..., None]).masked_fill(~seen[:, None], -math.inf))
    p = p.reshape(b, hk, -1, most).sum(2)
    old = st["weights"][:, :, :most]
    # committed tokens gather, new ones begin, what lies behind them stays
    st["weights"][:, :, :most] = torch.where(j < 0, old + p, torch.where(j < news, p, old))
    return {"weights": st["weights"]}


def _plain_evict(st):
    case = st["case"]
    b, hk, d, page = (case[x] for x in ("batch", "kv_heads", "head_dim", "page"))
    budget, recent, sink = case["budget"], case["recent"], case["sink"]
    w = st["weights"]
    t = torch.arange(w.shape[2], device="cuda")
    length = st["lengths"].long()[:, None, None]
    # in descending order of rank: the sinks and the latest tokens, the others by weight, lower places first
    rank = torch.where((t < sink) | (t >= length - recent), math.inf, w)
    rank = torch.where(t < length, rank, -math.inf)
    most = min(budget, w.shape[2])
    keep = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :most]
    count = length.clamp(max=budget)
    i = torch.arange(most, device="cuda")
    keep = torch.sort(torch.where(i < count, keep, w.shape[2]), dim=-1)[0]  # [b, hk, most], in order of place
    weights = torch.zeros((b, hk, st["to"].shape[1] * page), device="cuda")
    bb, hh, ii = torch.nonzero((i < count).expand(b, hk, most), as_tuple=True)
    src = keep[bb, hh, ii]
    weights[bb, hh, ii] = w[bb, hh, src]
    fro, to = st["table"].long()[bb, src // page], st["to"].long()[bb, ii // page]
    for pool in (st["k_pages"], st["v_pages"]):
        pool[to, hh, ii % page] = pool[fro, hh, src % page]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "weights": weights, "lengths": count[:, 0, 0].to(torch.int32)}


def _own(st):
    import block_sparse_attention_causal_gb300 as wise
    case, op = st["case"], st["case"]["op"]
    if op == "rotate":
        rope = wise.Rope(st["steps"], case["pairs"], st["axes"])
        q, k = wise.norm_rotate(st["q"], st["k"], q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=EPS,
                                positions=st["positions"], rope=rope)
        return {"q": q, "k": k}
    cache = wise.PagedCache(st["k_pages"], st["v_pages"], st["table"], st["lengths"])
    if op == "append":
        rope = wise.Rope(st["steps"], case["pairs"], st["axes"])
        q = wise.cache_append(cache, st["k"], st["v"], q=st["q"], new_len=st["new_len"], positions=st["positions"], rope=rope,
                              q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=EPS)
        out = {"k_pages": cache.k_pages, "v_pages": cache.v_pages}
        return out if q is None else dict(out, q=q)
    if op == "prefix":
        out, lse = wise.prefix_attention(st["q"], cache, st["prefix"], group_starts=st["starts"], new_len=st["new_len"],
                                         tree_mask=st["mask"])
        return {"out": out, "lse": lse}
    if op == "weights":
        return {"weights": wise.cache_weights(st["q"], cache, st["lse"], st["weights"], new_len=st["new_len"])}
    kept, weights = wise.cache_evict(cache, st["weights"], case["budget"], st["to"], recent=case["recent"], sink=case["sink"])
    return {"k_pages": kept.k_pages, "v_pages": kept.v_pages, "weights": weights, "lengths": kept.lengths}


def run(st):
    if own:
        return _own(st)
    return {"append": _plain_append, "rotate": _plain_rotate, "prefix": _plain_prefix, "weights": _plain_weights,
            "evict": _plain_evict}[st["case"]["op"]](st)


# ------------------------------------------------------------ in 64 bits

def _exact_rows(x, weight, turn, pairs):
    """x [heads, n, d] normed, then its first values times exp(i turn) as complex numbers; turn [n, r / 2]."""
    x = x.double()
    w = weight.double()
    x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * (w[:, None] if w.dim() == 2 else w)
    r = 2 * turn.shape[-1]
    z = x[..., :r]
    z = z.unflatten(-1, (r // 2, 2)) if pairs else z.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(turn), turn))
    y = y if pairs else y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., r:]], dim=-1)


def _exact_turn(st, i, start):
    n = st["case"]["new"]
    if st["positions"] is None:
        return torch.arange(start, start + n, device="cuda").double()[:, None] * st["inv_freq"][None]
    axes = st["axes"].tolist()
    return torch.stack([st["positions"][a, i].double() * st["inv_freq"][x] for x, a in enumerate(axes)], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        turns = [_exact_turn(st, i, 0) for i in range(case["batch"])]
        return {x: torch.stack([_exact_rows(st[x][i], st[x + "_norm"], turns[i], case["pairs"]) for i in range(case["batch"])])
                for x in ("q", "k")}
    lengths, news = _lengths(case)
    page, hk, d = case["page"], case["kv_heads"], case["head_dim"]
    table = st["table"].tolist()
    if op == "append":
        kp, vp, qs = st["k_pages"].double(), st["v_pages"].double(), []
        for b in range(case["batch"]):
            turn = _exact_turn(st, b, lengths[b])
            k, v = _exact_rows(st["k"][b], st["k_norm"], turn, case["pairs"]), st["v"][b].double()
            done = 0
            while done < news[b]:  # page by page
                slot = lengths[b] + done
                m = min(page - slot % page, news[b] - done)
                kp[table[b][slot // page], :, slot % page:slot % page + m] = k[:, done:done + m]
                vp[table[b][slot // page], :, slot % page:slot % page + m] = v[:, done:done + m]
                done += m
            if st["q"] is not None:
                qs.append(_exact_rows(st["q"][b], st["q_norm"], turn, case["pairs"]))
        out = {"k_pages": kp, "v_pages": vp}
        return dict(out, q=torch.stack(qs)) if qs else out
    if op == "evict":
        return _exact_evict(st, lengths, table)
    h, n = case["heads"], case["new"]
    b_ = len(lengths)
    line = []  # the new tokens that each one sees: itself and those above it, or all before it
    for i in range(n):
        line.append([i] if i == 0 else line[(i - 1) // case.get("branch", 1)] + [i])
    out = torch.zeros((b_, h, n, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b_, h, n), -math.inf, dtype=torch.float64, device="cuda")
    weights = st["weights"].double() if op == "weights" else None
    for b in range(b_):
        m, length = news[b], lengths[b]
        sees = torch.zeros((m, length + m), dtype=torch.bool)
        sees[:, :length] = True
        for i in range(m):
            sees[i, torch.tensor(line[i]) + length] = True
        sees = sees.cuda()
        pages = torch.tensor(table[b][:(length + m + page - 1) // page], device="cuda")
        for x in range(hk):
            k = st["k_pages"][pages, x].reshape(-1, d)[:length + m].double()
            mine = slice(x * (h // hk), (x + 1) * (h // hk))
            s = (st["q"][b, mine, :m].double() @ k.T) * d ** -0.5
            s = s.masked_fill(~sees, -math.inf)
            if op == "weights":
                p = torch.exp(s - st["lse"][b, mine, :m, None].double()).sum((0, 1))
                weights[b, x, :length] += p[:length]
                weights[b, x, length:length + m] = p[length:]
                continue
            v = st["v_pages"][pages, x].reshape(-1, d)[:length + m].double()
            lse[b, mine, :m] = torch.logsumexp(s, -1)
            out[b, mine, :m] = torch.exp(s - lse[b, mine, :m, None]) @ v
    return {"weights": weights} if op == "weights" else {"out": out, "lse": lse}


def _exact_evict(st, lengths, table):
    case = st["case"]
    hk, page, budget, recent, sink = (case[x] for x in ("kv_heads", "page", "budget", "recent", "sink"))
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    to = st["to"].tolist()
    weights = torch.zeros((len(lengths), hk, len(to[0]) * page), dtype=torch.float64, device="cuda")
    host = st["weights"].cpu()
    for b, length in enumerate(lengths):
        count = min(length, budget)
        row = torch.tensor(table[b], device="cuda")
        goes = torch.tensor(to[b], device="cuda")
        for x in range(hk):
            if length <= budget:
                keep = list(range(length))
            else:
                w = host[b, x].tolist()
                middle = sorted(range(sink, length - recent), key=lambda i: (-w[i], i))[:budget - recent - sink]
                keep = sorted(list(range(sink)) + middle + list(range(length - recent, length)))
            src, dst = torch.tensor(keep, dtype=torch.int64, device="cuda"), torch.arange(count, device="cuda")
            weights[b, x, :count] = st["weights"][b, x, src].double()
            for pool, old in ((kp, st["k_pages"]), (vp, st["v_pages"])):
                pool[goes[dst // page], x, dst % page] = old[row[src // page], x, src % page].double()
    return {"k_pages": kp, "v_pages": vp, "weights": weights, "lengths": None}
