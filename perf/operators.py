"""Workloads of the serving operators: keys and values appended to a paged
cache with the position rotation, attention of drafted token trees (and of
single tokens) over that cache, and the acceptance of a drafted path.

Sizes come from the library's own configurations (32 heads of 128, 40 heads
of 96, 2 heads of 64, grouped-query attention of 32 over 8 heads, contexts of
2K to 32K, pages of 16 to 128) or are generic serving sizes.
"""
import math
import random

import torch

own = False

TWO_PI = 2.0 * math.pi


# ------------------------------------------------------------------- cases

def _attend(name, batch, heads, kv_heads, head_dim, page, ctx, new, branch, ragged):
    c = dict(op="attend", batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, ctx=ctx, new=new,
             branch=branch, ragged=ragged)
    return dict(c, name=name) if name else c


def _append(name, batch, heads, kv_heads, head_dim, page, ctx, new, branch, ragged, rotary, interleaved, with_q):
    c = dict(op="append", batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, ctx=ctx, new=new,
             branch=branch, ragged=ragged, rotary=rotary, interleaved=interleaved, with_q=with_q)
    return dict(c, name=name) if name else c


def _accept(name, batch, kv_heads, head_dim, page, ctx, new, accepted, ragged):
    c = dict(op="accept", batch=batch, heads=kv_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, ctx=ctx,
             new=new, branch=1, accepted=accepted, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token behind a short prompt: latency counts
        _attend("token_2k", 1, 32, 8, 128, 64, 2048, 1, 1, False),
        # a small drafted tree behind a few hundred tokens, small heads, small pages
        _attend("tree_small_d64", 3, 8, 2, 64, 16, 333, 7, 2, True),
        # a full server's next tokens, sequences of different lengths
        _attend("token_batch_8k", 32, 32, 8, 128, 64, 8192, 1, 1, True),
        # one long conversation's next token
        _attend("token_128k", 1, 32, 8, 128, 128, 131071, 1, 1, False),
        # a drafted tree of 64 tokens behind 32K of context, grouped heads
        _attend("tree_64_32k", 1, 32, 8, 128, 128, 32768, 64, 3, False),
        # drafted trees of up to 13 tokens, every head with keys of its own, 96 wide
        _attend("tree_13_d96_16k", 2, 40, 40, 96, 32, 16384, 13, 2, True),
        # a prompt of 32K enters the cache, its queries rotated on the way
        _append("append_prompt_32k", 1, 32, 8, 128, 128, 0, 32768, 1, False, 128, False, True),
        # one token of each of 64 users
        _append("append_token_b64", 64, 32, 8, 128, 64, 8192, 1, 1, True, 128, False, True),
        # ragged drafted trees, neighbouring pairs rotated, three quarters of the head rotated
        _append("append_tree_d96", 8, 40, 40, 96, 16, 4096, 13, 2, True, 64, True, True),
        # one user's drafted path of 5 is kept
        _accept("accept_one", 1, 8, 128, 64, 4096, 64, 5, False),
        # 64 users keep up to 12 drafted tokens each
        _accept("accept_b64", 64, 8, 128, 32, 2048, 64, 12, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (32, 32, 128), (40, 40, 96), (8, 2, 64), (32, 4, 64), (40, 8, 96),
                                       (16, 1, 128), (2, 2, 64)])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    op = rng.choice(["attend", "attend", "append", "accept"])
    batch = _log(rng, 1, 64)
    if op == "attend":
        new, branch = _log(rng, 1, 128), rng.choice([1, 2, 3, 8])
        ctx = _log(rng, 1, 131072)
        case = lambda: _attend(None, batch, heads, kv_heads, dim, page, ctx, new, branch, ragged)  # noqa: E731
        most = work(listed()[2])
        while work(case())["bytes"] > most["bytes"] or work(case())["flops"] > 2e11 or batch * heads * new * ctx > 2 ** 28:
            if batch > 1 and rng.random() < 0.5:
                batch = (batch + 1) // 2
            else:
                ctx = max(1, ctx // 2)
                new = max(1, new - new // 8)
        return case()
    if op == "append":
        new, branch, ctx = _log(rng, 1, 32768), rng.choice([1, 2, 3]), rng.choice([0, _log(rng, 1, 32768)])
        rotary = rng.choice([dim, dim // 2, 0, 32])
        inter, with_q = rng.random() < 0.5, rng.random() < 0.6
        case = lambda: _append(None, batch, heads, kv_heads, dim, page, ctx, new, branch, ragged, rotary, inter, with_q)  # noqa: E731
        while work(case())["bytes"] > 8e8 or batch * (ctx + new) * kv_heads > 2 ** 21:
            if batch > 1 and rng.random() < 0.5:
                batch = (batch + 1) // 2
            else:
                new, ctx = max(1, new // 2), ctx // 2
        return case()
    new = _log(rng, 4, 128)
    accepted = rng.randint(2, max(2, new // 2))
    ctx = _log(rng, 1, 4096)
    return _accept(None, batch, kv_heads, dim, page, ctx, new, accepted, ragged)


def _lengths(case):
    """Committed tokens and new tokens of each sequence."""
    b, ctx, new = case["batch"], case["ctx"], case["new"]
    if not case["ragged"]:
        return [ctx] * b, [new] * b
    lengths = [max(0, ctx - (ctx * ((5 * i) % 8)) // 9 - i % 3) for i in range(b)]
    return lengths, [max(1, new - (new * (i % 4)) // 4) for i in range(b)]


def _accepted(case):
    """Accepted tokens of each sequence, at most half of its drafted ones."""
    a, news = case["accepted"], _lengths(case)[1]
    return [min(max(1, y // 2), a if not case["ragged"] else max(1, a - (a * (i % 3)) // 3)) for i, y in enumerate(news)]


def _depths(case, most):
    """Depth of each drafted token: token i hangs below token (i - 1) // branch, the first below the context."""
    depth = [0] * most
    for i in range(1, most):
        depth[i] = depth[(i - 1) // case["branch"]] + 1
    return depth


def work(case):
    lengths, news = _lengths(case)
    hk, h, d, n = case["kv_heads"], case["heads"], case["head_dim"], case["new"]
    if case["op"] == "attend":
        keys = sum(x + y for x, y in zip(lengths, news))
        depth = _depths(case, n)
        pairs = sum(x * y + sum(depth[:y]) + y for x, y in zip(lengths, news))
        nbytes = keys * hk * d * 4 + sum(news) * h * d * 2 + case["batch"] * n * h * (d * 2 + 4)
        return {"bytes": nbytes, "flops": 4 * d * h * pairs}
    if case["op"] == "append":
        tokens = sum(news)
        nbytes = tokens * hk * d * 8 + (case["batch"] * n * h * d * 4 if case["with_q"] else 0)
        return {"bytes": nbytes, "flops": 3 * case["rotary"] * (tokens * hk + (case["batch"] * n * h if case["with_q"] else 0))}
    moved = sum(a - 1 for a in _accepted(case))  # the first drafted token stays where it is
    return {"bytes": max(moved, 1) * hk * d * 8, "flops": 0}


# ------------------------------------------------------------------ inputs

def _mask_words(case):
    """[n, ceil(n / 32)] int32: bit j % 32 of word j // 32 of row i: drafted token i sees drafted token j."""
    n = case["new"]
    rows = []
    for i in range(n):
        bits = (1 << i) | (rows[(i - 1) // case["branch"]] if i else 0)
        rows.append(bits)
    words = [[(r >> (32 * w)) & 0xffffffff for w in range((n + 31) // 32)] for r in rows]
    return torch.tensor([[x - (1 << 32) if x >> 31 else x for x in r] for r in words], dtype=torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    b, h, hk, d, n, page = (case[x] for x in ("batch", "heads", "kv_heads", "head_dim", "new", "page"))
    lengths, news = _lengths(case)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(torch.bfloat16)

    used = [(x + y + page - 1) // page for x, y in zip(lengths, news)]
    max_pages = max(used) + 1
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    starts = torch.tensor([sum(used[:i]) for i in range(b)], device=dev)
    held = torch.tensor(used, device=dev)
    col = torch.arange(max_pages, device=dev)
    table = torch.where(col[None] < held[:, None], order[(starts[:, None] + col[None]).clamp(max=n_pages - 1)], -1).to(torch.int32)
    st = dict(case=case, k_pages=normal(n_pages, hk, page, d), v_pages=normal(n_pages, hk, page, d), table=table,
              lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
              new_len=torch.tensor(news, dtype=torch.int32, device=dev) if case["ragged"] else None)
    if case["op"] == "attend":
        # queries and keys of a few units' length: some keys stand out
        st["q"] = normal(b, h, n, d, scale=1.5)
        st["mask"] = None if case["branch"] == 1 else _mask_words(case).to(dev)[None].expand(b, -1, -1).contiguous()
        st["news"] = torch.tensor(news, dtype=torch.int32, device=dev)
    elif case["op"] == "append":
        # one projection's output holds queries, keys and values of a token side by side
        qkv = normal(b, n, h + 2 * hk, d)
        qkv = qkv.transpose(1, 2)
        st["q"] = qkv[:, :h] if case["with_q"] else None
        st["k"], st["v"] = qkv[:, h:h + hk], qkv[:, h + hk:]
        r = case["rotary"]
        inv_freq = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
        st["inv_freq"] = torch.tensor(inv_freq, dtype=torch.float64, device=dev)
        # turns per position in units of 2^-64, as signed 64-bit whole numbers
        steps = [int(round(f / TWO_PI * 2.0 ** 64)) for f in inv_freq]
        st["steps"] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in steps], dtype=torch.int64, device=dev)
        st["positions"] = None
        if case["branch"] > 1:
            depth = torch.tensor(_depths(case, n), dtype=torch.int32, device=dev)
            st["positions"] = (st["lengths"][:, None] + depth[None]).contiguous()
        i = torch.arange(n, device=dev)
        st["token"] = torch.nonzero(i[None] < torch.tensor(news, device=dev)[:, None], as_tuple=True)
    else:
        kept = _accepted(case)
        a = max(kept)
        st["n_accepted"] = torch.tensor(kept, dtype=torch.int32, device=dev)
        rng = random.Random(seed)
        # the first drafted token, then tokens behind the first few of a broad tree
        path = [[0] + sorted(rng.sample(range(x, news[i]), x - 1)) + [-1] * (a - x) for i, x in enumerate(kept)]
        st["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
        i = torch.arange(a, device=dev)
        st["token"] = torch.nonzero(i[None] < st["n_accepted"][:, None], as_tuple=True)
    return st


# -------------------------------------------------------------- plain forms

def _slots(st, batch, token):
    """Page and row of token `token` behind the committed ones of sequence `batch`."""
    page = st["k_pages"].shape[2]
    pos = st["lengths"].long()[batch] + token
    return st["table"].long()[batch, pos // page], pos % page


def _rotate(x, angle, interleaved):
    """x [..., d] in 32 bits, angle [..., r / 2] in 64 bits: the first r values of each head, in pairs."""
    half = angle.shape[-1]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2), rest], dim=-1)
    a, b = rot[..., :half], rot[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], dim=-1)


def _plain_append(st):
    case = st["case"]
    n = case["new"]
    at = st["positions"] if st["positions"] is not None else st["lengths"][:, None] + torch.arange(n, device="cuda")
    angle = at.double()[..., None] * st["inv_freq"]  # [batch, n, r / 2]
    b, i = st["token"]
    page, row = _slots(st, b, i)
    k = st["k"][b, :, i].float()  # [tokens, kv_heads, d]
    st["k_pages"][page, :, row] = _rotate(k, angle[b, i][:, None], case["interleaved"]).to(torch.bfloat16)
    st["v_pages"][page, :, row] = st["v"][b, :, i]
    out = {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if st["q"] is not None:
        out["q"] = _rotate(st["q"].float(), angle[:, None], case["interleaved"]).to(torch.bfloat16)
    return out


def _plain_attend(st):
    case = st["case"]
    b, h, hk, d, n = (case[x] for x in ("batch", "heads", "kv_heads", "head_dim", "new"))
    table = st["table"].long()
    k = st["k_pages"][table].transpose(1, 2).reshape(b, hk, -1, d).float()
    v = st["v_pages"][table].transpose(1, 2).reshape(b, hk, -1, d).float()
    key = torch.arange(k.shape[2], device="cuda")
    length, news = st["lengths"].long()[:, None, None], st["news"].long()[:, None, None]
    j = key[None, None] - length  # [batch, 1, keys]: drafted token of a key behind the committed ones
    row = torch.arange(n, device="cuda")[None, :, None]
    if st["mask"] is None:
        sees = j <= row
    else:
        at = j.clamp(0, n - 1).expand(b, n, -1)
        sees = (torch.gather(st["mask"], 2, at // 32) >> (at % 32).int()) & 1 == 1
    seen = (row < news) & ((j < 0) | ((j < news) & sees))  # [batch, n, keys]
    s = st["q"].float().reshape(b, hk, -1, d) @ k.transpose(2, 3) / math.sqrt(d)
    s = s.reshape(b, h, n, -1).masked_fill(~seen[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(b, hk, -1, p.shape[-1]) @ v).reshape(b, h, n, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.log(total[..., 0]) + torch.where(torch.isinf(top), 0.0, top)[..., 0]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_accept(st):
    b, i = st["token"]
    page, row = _slots(st, b, st["path"].long()[b, i])
    to_page, to_row = _slots(st, b, i)
    st["k_pages"][to_page, :, to_row] = st["k_pages"][page, :, row]
    st["v_pages"][to_page, :, to_row] = st["v_pages"][page, :, row]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "lengths": st["lengths"] + st["n_accepted"]}


def run(st):
    op = st["case"]["op"]
    if own:
        import block_sparse_attention_causal_gb300 as wise
        cache = wise.PagedCache(st["k_pages"], st["v_pages"], st["table"], st["lengths"])
        if op == "attend":
            out, lse = wise.tree_attention(st["q"], cache, new_len=st["new_len"], tree_mask=st["mask"])
            return {"out": out, "lse": lse}
        if op == "append":
            rope = wise.Rope(st["steps"], st["case"]["interleaved"])
            q = wise.cache_append(cache, st["k"], st["v"], q=st["q"], new_len=st["new_len"], positions=st["positions"],
                                  rope=rope)
            out = {"k_pages": cache.k_pages, "v_pages": cache.v_pages}
            return out if q is None else dict(out, q=q)
        lengths = wise.cache_accept(cache, st["n_accepted"], st["path"])
        return {"k_pages": cache.k_pages, "v_pages": cache.v_pages, "lengths": lengths}
    return {"attend": _plain_attend, "append": _plain_append, "accept": _plain_accept}[op](st)


# ------------------------------------------------------------ in 64 bits

def _complex_rotation(x, turn, interleaved):
    """x [..., d] times exp(i turn) on pairs of its first values, as complex numbers in 64 bits."""
    r = 2 * turn.shape[-1]
    if r == 0:
        return x
    z = x[..., :r]
    z = z.unflatten(-1, (r // 2, 2)) if interleaved else z.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(turn), turn))
    w = w if interleaved else w.transpose(-1, -2)
    return torch.cat([w.flatten(-2), x[..., r:]], dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    lengths, news = _lengths(case)
    page, n = case["page"], case["new"]
    table = st["table"].tolist()
    if case["op"] == "accept":
        out = {"k_pages": st["k_pages"].double(), "v_pages": st["v_pages"].double()}
        path = st["path"].tolist()
        for b, a in enumerate(_accepted(case)):
            for i in range(a):
                x, y = lengths[b] + path[b][i], lengths[b] + i
                for pool in (out["k_pages"], out["v_pages"]):
                    pool[table[b][y // page], :, y % page] = pool[table[b][x // page], :, x % page].clone()
        return dict(out, lengths=None)
    if case["op"] == "append":
        kp, vp = st["k_pages"].double(), st["v_pages"].double()
        turn = []
        for b in range(case["batch"]):
            at = torch.arange(lengths[b], lengths[b] + n, device="cuda") if st["positions"] is None else st["positions"][b]
            turn.append(at.double()[:, None] * st["inv_freq"][None])
            k = _complex_rotation(st["k"][b].double(), turn[b][None], case["interleaved"])
            v = st["v"][b].double()
            done = 0
            while done < news[b]:  # page by page
                slot = lengths[b] + done
                m = min(page - slot % page, news[b] - done)
                kp[table[b][slot // page], :, slot % page:slot % page + m] = k[:, done:done + m]
                vp[table[b][slot // page], :, slot % page:slot % page + m] = v[:, done:done + m]
                done += m
        out = {"k_pages": kp, "v_pages": vp}
        if st["q"] is not None:
            out["q"] = torch.stack([_complex_rotation(st["q"][b].double(), turn[b][None], case["interleaved"]) for b in range(case["batch"])])
        return out
    b_, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
    out = torch.zeros((b_, h, n, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b_, h, n), -math.inf, dtype=torch.float64, device="cuda")
    line = []  # the drafted tokens that each one sees: itself and those above it, or all before it
    for i in range(n):
        line.append([i] if i == 0 else line[(i - 1) // case["branch"]] + [i])
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
            v = st["v_pages"][pages, x].reshape(-1, d)[:length + m].double()
            for y in range(x * (h // hk), (x + 1) * (h // hk)):
                s = (st["q"][b, y, :m].double() @ k.T) * d ** -0.5
                s = s.masked_fill(~sees, -math.inf)
                lse[b, y, :m] = torch.logsumexp(s, -1)
                out[b, y, :m] = torch.exp(s - lse[b, y, :m, None]) @ v
    return {"out": out, "lse": lse}
