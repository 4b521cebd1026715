"""Cases of the operators for requests that share pages of the latent cache.

  shared   absorbed attention of a batch whose requests share long prefixes: a
           prefix is read once for all requests of its group
  fork     requests that go on from another request's tokens: whole pages are
           shared, the rows of a page that is not full are copied
  release  pages that nobody holds any more, after requests have ended or
           dropped their last tokens
  compact  held pages together at the start of the cache
  copy     pages from one cache into another

Rows of the cache are 512 latent and 64 key values (bf16), lengths, page ids and
the counts of holders int32.  `shares` counts the holders of a page beyond the
first: a page that one request holds has 0.
"""
import math
import random

import torch

own = False

LAT, PE = 512, 64
ROW = LAT + PE
SCALE = 192 ** -0.5
NO_PAGE = 0  # what a table holds behind a request's last page


# ---- cases ----

def listed():
    return [
        # a few samples of one prompt of a chat: latency
        dict(name="shared_samples", op="shared", groups=1, members=8, heads=16, new=1, prefix=1024, tail=128, ragged=False, page=64, lens=1),
        # a serving batch behind one system prompt
        dict(name="shared_system", op="shared", groups=1, members=256, heads=32, new=1, prefix=4096, tail=512, ragged=True, page=64, lens=2),
        # prompts of several users, each with a few samples, lengths of all sorts, small pages
        dict(name="shared_users", op="shared", groups=24, members=16, heads=16, new=1, prefix=8192, tail=1024, ragged=True, page=16, lens=3),
        # questions to two long documents, three drafted tokens each
        dict(name="shared_documents", op="shared", groups=2, members=24, heads=32, new=3, prefix=49152, tail=256, ragged=False, page=128, lens=4),
        # one prompt's samples start
        dict(name="fork_samples", op="fork", parents=1, children=8, cached=1000, whole=True, page=16, lens=5),
        # a batch of prompts with sixteen samples each, from any place of the prompt
        dict(name="fork_batch", op="fork", parents=16, children=256, cached=8192, whole=False, page=64, lens=6),
        # requests of a decoding batch that have ended
        dict(name="release_ended", op="release", requests=256, rows=16, cached=4096, family=1, keep=False, page=64, lens=7),
        # all samples of a long batch drop part of what they hold, small pages
        dict(name="release_branches", op="release", requests=256, rows=256, cached=16384, family=8, keep=True, page=16, lens=8),
        # a small cache before it is saved
        dict(name="compact_small", op="compact", requests=8, cached=512, family=2, spare=0.5, page=16, lens=9),
        # half of a large cache has become free
        dict(name="compact_large", op="compact", requests=64, cached=4096, family=4, spare=1.0, page=64, lens=10),
        # one request's pages to another cache
        dict(name="copy_request", op="copy", pages=33, page=64, spare=1.0),
        # a prefill worker's pages to the cache that decoding reads
        dict(name="copy_batch", op="copy", pages=8000, page=16, spare=0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "fork", "release", "compact", "copy"])
    seed = rng.randrange(1 << 20)
    page = rng.choice([8, 16, 16, 32, 48, 64, 64, 128, 256])
    if op == "shared":
        heads = rng.choice([1, 4, 8, 12, 16, 24, 32, 40, 64, 128])
        new = rng.choice([1, 1, 1, 2, 3])
        groups = _log(rng, 1, 32)
        members = _log(rng, 1, max(1, 256 // groups))
        prefix = _log(rng, 1, 65536)
        tail = _log(rng, new, 2048)
        # query rows times tokens, and tokens, stay within the largest listed case's
        rows = groups * members * heads * new
        while rows * (prefix + tail) > 2 * 24 * 32 * 3 * 49152 or groups * (prefix + members * tail) > 1 << 18:
            prefix, tail = max(1, prefix // 2), max(new, tail // 2)
        return dict(op=op, groups=groups, members=members, heads=heads, new=new, prefix=prefix, tail=tail,
                    ragged=rng.random() < 0.7, page=page, lens=seed)
    if op == "fork":
        parents = _log(rng, 1, 16)
        return dict(op=op, parents=parents, children=_log(rng, 1, 256), cached=_log(rng, 1, 8192), whole=rng.random() < 0.5,
                    page=page, lens=seed)
    if op == "release":
        requests = _log(rng, 1, 256)
        return dict(op=op, requests=requests, rows=_log(rng, 1, requests), cached=_log(rng, 1, 16384),
                    family=rng.choice([1, 2, 3, 8]), keep=rng.random() < 0.5, page=max(16, page), lens=seed)
    if op == "compact":
        return dict(op=op, requests=_log(rng, 1, 64), cached=_log(rng, 1, 4096), family=rng.choice([1, 2, 4]),
                    spare=rng.choice([0.0, 0.1, 0.5, 1.0]), page=page, lens=seed)
    return dict(op=op, pages=_log(rng, 1, 128000 // page), page=page, spare=rng.choice([0.0, 0.3, 1.0]))


def _pages(tokens, page):
    return -(-tokens // page)


def _shared_lengths(case):
    """Requests of each group, prefix of each group, tokens behind it of each request; all by the case alone."""
    rng = random.Random(case["lens"])
    ragged = case["ragged"]
    members = [case["members"] if g == 0 or not ragged else rng.randint(1, case["members"]) for g in range(case["groups"])]
    prefix = [case["prefix"] if g == 0 or not ragged else rng.randint(1, case["prefix"]) for g in range(case["groups"])]
    tail = [case["tail"] if b == 0 or not ragged else rng.randint(case["new"], case["tail"]) for b in range(sum(members))]
    return members, prefix, tail


def _fork_lengths(case):
    """Tokens of each parent, the parent of each child, and how many of its tokens the child takes."""
    rng = random.Random(case["lens"])
    cached = [case["cached"] if p == 0 else rng.randint(1, case["cached"]) for p in range(case["parents"])]
    of = [rng.randrange(case["parents"]) for _ in range(case["children"])]
    return cached, of, [cached[p] if case["whole"] else rng.randint(1, cached[p]) for p in of]


def _family_lengths(case):
    """Tokens of each request, and how many of them the requests of its family share (a number of whole pages)."""
    rng = random.Random(case["lens"])
    n, page, family = case["requests"], case["page"], case["family"]
    cached = [case["cached"] if b == 0 else rng.randint(1, case["cached"]) for b in range(n)]
    common = []
    for b in range(0, n, family):
        shortest = min(cached[b:b + family])
        common += [rng.randint(0, shortest // page) if family > 1 else 0] * len(cached[b:b + family])
    return cached, common


def _release_rows(case, cached):
    rng = random.Random(case["lens"] + 1)
    rows = rng.sample(range(case["requests"]), case["rows"])
    return rows, [rng.randint(0, cached[b]) if case["keep"] else 0 for b in rows]


# ---- inputs ----

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 29)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    def perm(n):
        return torch.randperm(n, generator=gen, device=dev).to(torch.int32)

    def tables(common, held, first, width, ids):
        """Rows of page ids: `common` pages from place first[b] of `ids`, which several rows may have, then the row's own."""
        common, held, first = ints(common), ints(held), ints(first)
        mine = held - common
        start = ids.numel() - int(mine.sum()) + mine.cumsum(0) - mine
        col = torch.arange(width, device=dev)[None, :]
        at = torch.where(col < common[:, None], first[:, None] + col, start[:, None] + col - common[:, None])
        table = ids[at.clamp(0, max(0, ids.numel() - 1)).long()]
        return torch.where(col < held[:, None], table, torch.full_like(table, NO_PAGE))

    op, page = case["op"], case["page"]
    state = {"case": case}
    if op == "shared":
        members, prefix, tail = _shared_lengths(case)
        group = [g for g, m in enumerate(members) for _ in range(m)]
        lens = [prefix[g] + t for g, t in zip(group, tail)]
        common = [prefix[g] // page for g in group]
        held = [_pages(n, page) for n in lens]
        starts = [sum(x // page for x in prefix[:g]) for g in range(len(prefix))]
        total = sum(x // page for x in prefix) + sum(h - c for h, c in zip(held, common))
        n = len(lens)
        pages = total + 3
        table = tables(common, held, [starts[g] for g in group], max(held), perm(pages)[:total])
        cache = normal(pages, page, ROW)
        # the prefix's last rows, in a page that is not full: every request has its own copy of them
        first = [group.index(g) for g in group]
        at = torch.tensor(common, device=dev)
        mine = table[torch.arange(n, device=dev), at.clamp(max=max(held) - 1)].long()
        part = torch.arange(page, device=dev)[None, :, None] < ints([prefix[g] % page for g in group])[:, None, None]
        cache[mine] = torch.where(part, cache[mine[torch.tensor(first, device=dev)]], cache[mine])
        state.update(q=normal(n, case["new"], case["heads"], ROW), cache=cache, table=table, lens=ints(lens),
                     cu=torch.tensor([0] + members, device=dev).cumsum(0), prefix=ints(prefix), scale=SCALE,
                     most=(max(members), max(prefix), max(tail)), group=torch.tensor(group, device=dev),
                     lse=torch.empty((n, case["new"], case["heads"]), dtype=torch.float32, device=dev))
    elif op == "fork":
        cached, of, take = _fork_lengths(case)
        held = [_pages(x, page) for x in cached]
        requests = len(cached) + len(of)
        pages = sum(held) + len(of) + 3
        ids = perm(pages)
        width = max(held) + 1
        order = torch.randperm(requests, generator=gen, device=dev)  # rows of the table: parents, then children
        table = torch.full((requests, width), NO_PAGE, dtype=torch.int32, device=dev)
        table[order[:len(cached)]] = tables([0] * len(cached), held, [0] * len(cached), width, ids[:sum(held)])
        lens = torch.zeros(requests, dtype=torch.int32, device=dev)
        lens[order[:len(cached)]] = ints(cached)
        state.update(parents=order[torch.tensor(of, device=dev)].to(torch.int32), children=order[len(cached):].to(torch.int32),
                     take=None if case["whole"] else ints(take), table=table, lens=lens, free=ids[sum(held):].contiguous(),
                     shares=torch.zeros(pages, dtype=torch.int32, device=dev), cache=normal(pages, page, ROW), page=page)
    elif op in ("release", "compact"):
        cached, common = _family_lengths(case)
        n, family = case["requests"], case["family"]
        held = [_pages(x, page) for x in cached]
        first, place = [], 0
        for b in range(0, n, family):
            first += [place] * len(cached[b:b + family])
            place += common[b]
        total = place + sum(h - c for h, c in zip(held, common))
        pages = total + int(total * case.get("spare", 0.25)) + 2
        ids = perm(pages)[:total]
        table = tables(common, held, first, max(held) + 1, ids)
        shares = torch.zeros(pages, dtype=torch.int32, device=dev)
        col = torch.arange(table.shape[1], device=dev)[None, :] < ints(held)[:, None]
        shares = torch.bincount(table[col].long(), minlength=pages).sub_(1).clamp_(min=0).to(torch.int32)
        state.update(table=table, lens=ints(cached), shares=shares, page=page)
        if op == "release":
            rows, keep = _release_rows(case, cached)
            state.update(rows=ints(rows), keep=ints(keep) if case["keep"] else None)
        else:
            state.update(cache=normal(pages, page, ROW))
    else:
        n = case["pages"]
        src, dst = n + int(n * case["spare"]), n + int(n * case["spare"]) + 1
        state.update(src=normal(src, page, ROW), dst=normal(dst, page, ROW), src_pages=perm(src)[:n].contiguous(),
                     dst_pages=perm(dst)[:n].contiguous())
    return state


# ---- one pass ----

def run(state):
    return {"shared": _run_shared, "fork": _run_fork, "release": _run_release, "compact": _run_compact,
            "copy": _run_copy}[state["case"]["op"]](state)


def _run_shared(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_decode_shared
        out = latent_decode_shared(s["q"], s["cache"], s["table"], s["lens"], s["cu"], s["prefix"], s["scale"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    q, cache, table, cu, group = s["q"], s["cache"], s["table"], s["cu"], s["group"]
    n, new, heads, _ = q.shape
    page, dev = cache.shape[1], q.device
    members, longest, tail = s["most"]
    # prefixes: the requests of a group side by side, padded to the most, against the rows of its first request
    col = torch.arange(longest, device=dev)
    where = table[cu[:-1]][:, col // page].long()  # [groups, tokens]
    known = col[None, :] < s["prefix"][:, None]
    common = torch.where(known[..., None], cache[where, col % page].float(), torch.zeros((), device=dev))
    place = torch.arange(n, device=dev) - cu[group]
    side = torch.zeros((cu.numel() - 1, members, new * heads, ROW), device=dev)
    side[group, place] = q.reshape(n, new * heads, ROW).float()
    scores = torch.matmul(side.view(-1, members * new * heads, ROW), common.transpose(1, 2)).mul_(s["scale"])
    scores = scores.masked_fill_(~known[:, None, :], -math.inf).view(-1, members, new * heads, longest)[group, place]
    # the tokens behind them, by request
    step = torch.arange(tail, device=dev)[None, :]
    pos = s["prefix"][group].long()[:, None] + step
    there = pos < s["lens"].long()[:, None]
    safe = torch.where(there, pos, torch.zeros_like(pos))
    rows = cache[torch.gather(table, 1, safe // page).long(), safe % page].float()
    rows = torch.where(there[..., None], rows, torch.zeros((), device=dev))
    seen = s["lens"].long()[:, None] - (new - 1) + torch.arange(new, device=dev)[None, :]
    more = torch.matmul(q.reshape(n, new * heads, ROW).float(), rows.transpose(1, 2)).mul_(s["scale"])
    hidden = pos[:, None, None, :] >= seen[:, :, None, None]
    more = more.view(n, new, heads, tail).masked_fill_(hidden, -math.inf).view(n, new * heads, tail)
    top = torch.maximum(scores.amax(-1, keepdim=True), more.amax(-1, keepdim=True))
    scores, more = scores.sub_(top).exp_(), more.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True) + more.sum(-1, keepdim=True)
    side = torch.zeros((cu.numel() - 1, members, new * heads, longest), device=dev)
    side[group, place] = scores
    out = torch.matmul(side.view(-1, members * new * heads, longest), common[..., :LAT])
    out = out.view(-1, members, new * heads, LAT)[group, place] + torch.matmul(more, rows[..., :LAT])
    s["lse"].copy_((top + torch.log(total)).view(n, new, heads))
    return {"out": (out / total).view(n, new, heads, LAT).to(torch.bfloat16), "lse": s["lse"]}


def _run_fork(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_fork
        p = latent_fork(s["parents"], s["children"], s["lens"], s["table"], s["free"], s["shares"], s["cache"], s["take"])
        return {"table": s["table"], "shares": s["shares"], "cache": s["cache"], "seq_lens": p["seq_lens"],
                "pages_taken": p["pages_taken"]}
    page, table, cache = s["page"], s["table"], s["cache"]
    parents, children = s["parents"].long(), s["children"].long()
    take = (s["lens"][parents] if s["take"] is None else s["take"]).long()
    full, rest = take // page, take % page
    shared = torch.arange(table.shape[1], device=table.device)[None, :] < full[:, None]
    rows = table[parents]
    s["shares"].index_add_(0, rows[shared].long(), torch.ones((), dtype=torch.int32, device=table.device).expand(int(full.sum())))
    table[children] = torch.where(shared, rows, table[children])
    part = (rest > 0).nonzero().squeeze(1)
    fresh = s["free"][:part.numel()]
    table[children[part], full[part]] = fresh
    old, fresh = rows[part, full[part]].long(), fresh.long()
    kept = torch.arange(page, device=table.device)[None, :, None] < rest[part][:, None, None]
    cache[fresh] = torch.where(kept, cache[old], cache[fresh])
    lens = s["lens"].clone()
    lens[children] = take.to(torch.int32)
    return {"table": table, "shares": s["shares"], "cache": cache, "seq_lens": lens,
            "pages_taken": torch.full((1,), part.numel(), dtype=torch.int32, device=table.device)}


def _run_release(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_release
        p = latent_release(s["rows"], s["lens"], s["table"], s["shares"], s["page"], s["keep"])
        return {"shares": s["shares"], "seq_lens": p["seq_lens"], "pages": p["pages"], "count": p["count"]}
    page, table, shares, rows = s["page"], s["table"], s["shares"], s["rows"].long()
    keep = torch.zeros_like(s["rows"]) if s["keep"] is None else s["keep"]
    held = (s["lens"][rows] + page - 1) // page
    stays = (keep + page - 1) // page
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    dropped = table[rows][(col >= stays[:, None]) & (col < held[:, None])].long()
    left = shares - torch.bincount(dropped, minlength=shares.numel()).to(torch.int32)
    free = (left < 0).nonzero().squeeze(1).to(torch.int32)
    shares.copy_(left.clamp_(min=0))
    pages = torch.full_like(shares, -1)
    pages[:free.numel()] = free
    lens = s["lens"].clone()
    lens[rows] = keep
    return {"shares": shares, "seq_lens": lens, "pages": pages,
            "count": torch.full((1,), free.numel(), dtype=torch.int32, device=table.device)}


def _run_compact(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_compact
        p = latent_compact(s["lens"], s["table"], s["shares"], s["cache"])
        return {"cache": s["cache"], "table": p["block_table"], "shares": p["shares"], "page_map": p["page_map"],
                "pages_used": p["pages_used"]}
    page, table, shares, cache = s["page"], s["table"], s["shares"], s["cache"]
    held = torch.arange(table.shape[1], device=table.device)[None, :] < ((s["lens"] + page - 1) // page)[:, None]
    used = torch.zeros_like(shares, dtype=torch.bool)
    used[table[held].long()] = True
    count = used.sum()
    place = torch.arange(shares.numel(), device=table.device)
    movers, holes = (used & (place >= count)).nonzero().squeeze(1), (~used & (place < count)).nonzero().squeeze(1)
    cache[holes] = cache[movers]
    new = torch.where(used, place, torch.full_like(place, -1))
    new[movers] = holes
    counts = torch.where(used & (place < count), shares, torch.zeros_like(shares))
    counts[holes] = shares[movers]
    ids = torch.where(held, table, torch.zeros_like(table)).long()
    return {"cache": cache, "table": torch.where(held, new[ids].to(torch.int32), table), "shares": counts,
            "page_map": new.to(torch.int32), "pages_used": count.to(torch.int32).reshape(1)}


def _run_copy(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_copy
        return latent_copy(s["src"], s["src_pages"], s["dst"], s["dst_pages"])
    s["dst"][s["dst_pages"].long()] = s["src"][s["src_pages"].long()]
    return s["dst"]


# ---- what a pass cannot do without ----

def work(case):
    op, page = case["op"], case["page"]
    if op == "shared":
        members, prefix, tail = _shared_lengths(case)
        rows = case["heads"] * case["new"]
        group = [g for g, m in enumerate(members) for _ in range(m)]
        lens = [prefix[g] + t for g, t in zip(group, tail)]
        ids = sum(_pages(x, page) for x in prefix) + sum(_pages(n, page) - prefix[g] // page for g, n in zip(group, lens))
        moved = 2 * ROW * (sum(prefix) + sum(tail)) + 4 * ids + 4 * len(lens) + 12 * len(members)
        seen = sum(n - i for n in lens for i in range(case["new"])) * case["heads"]
        return {"bytes": moved + len(lens) * rows * (2 * ROW + 2 * LAT + 4), "flops": 2 * (ROW + LAT) * seen}
    if op == "fork":
        cached, _, take = _fork_lengths(case)
        ids = sum(x // page for x in take)
        copied = sum(x % page for x in take)
        # table entries and counts in and out, lengths, the children's and parents' numbers, rows copied
        return {"bytes": 16 * ids + 12 * len(take) + 8 * (len(cached) + len(take)) + 4 * ROW * copied, "flops": 0}
    if op in ("release", "compact"):
        cached, common = _family_lengths(case)
        held = [_pages(x, page) for x in cached]
        total = sum(common[b] for b in range(0, len(cached), case["family"])) + sum(h - c for h, c in zip(held, common))
        pages = total + int(total * case.get("spare", 0.25)) + 2
        if op == "release":
            rows, keep = _release_rows(case, cached)
            ids = sum(held[b] - _pages(k, page) for b, k in zip(rows, keep))
            return {"bytes": 4 * ids + 8 * len(rows) + 8 * len(cached) + 12 * pages, "flops": 0}
        # tables in and out, counts in and out, the map; on average as many pages move as lie behind the place of the last
        moves = total * (pages - total) / pages
        return {"bytes": 8 * sum(held) + 4 * len(cached) + 12 * pages + 4 * ROW * page * moves, "flops": 0}
    return {"bytes": case["pages"] * (4 * ROW * page + 8), "flops": 0}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op == "shared":  # every request for itself, over the rows that its own table names
        q, n, new, heads = s["q"], s["q"].shape[0], case["new"], case["heads"]
        out = torch.zeros((n, new, heads, LAT), dtype=torch.float64, device=q.device)
        lse = torch.full((n, new, heads), -math.inf, dtype=torch.float64, device=q.device)
        for b, length in enumerate(s["lens"].tolist()):
            rows = s["cache"][s["table"][b, :_pages(length, page)].long()].reshape(-1, ROW)[:length].double()
            for i in range(new):
                seen = length - (new - 1 - i)
                if seen > 0:
                    x = s["scale"] * (q[b, i].double() @ rows[:seen].T)
                    lse[b, i] = torch.logsumexp(x, 1)
                    out[b, i] = torch.softmax(x, 1) @ rows[:seen, :LAT]
        return {"out": out, "lse": lse}
    if op == "release":  # whole numbers: no value in 64 bits to be compared with
        return None
    if op == "fork":
        cache, free = s["cache"].double(), s["free"].tolist()
        table, lens = s["table"].tolist(), s["lens"].tolist()
        takes = [lens[p] for p in s["parents"].tolist()] if s["take"] is None else s["take"].tolist()
        taken = 0
        for parent, take in zip(s["parents"].tolist(), takes):
            if take % page:
                cache[free[taken], :take % page] = cache[table[parent][take // page], :take % page]
                taken += 1
        return {"cache": cache, "pages_taken": None, "seq_lens": None, "shares": None, "table": None}
    if op == "compact":
        cache, lens, table = s["cache"].double(), s["lens"].tolist(), s["table"].tolist()
        held = {p for b, length in enumerate(lens) for p in table[b][:_pages(length, page)]}
        count = len(held)
        moves = zip([p for p in range(count) if p not in held], sorted(p for p in held if p >= count))
        for to, at in moves:
            cache[to] = cache[at]
        return {"cache": cache, "page_map": None, "pages_used": None, "shares": None, "table": None}
    dst = s["dst"].double()
    for at, to in zip(s["src_pages"].tolist(), s["dst_pages"].tolist()):
        dst[to] = s["src"][at].double()
    return dst
