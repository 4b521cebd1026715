"""Cases of the latent-attention operators: the serving side of a full-attention
layer that keeps one shared latent vector a token in a paged cache.

  plan     block tables and slot maps from request lengths
  append   new tokens' latents (RMS-normalised) and key parts into the paged cache
  decode   absorbed form: the newest token(s) of every request against the cache
  prefill  expanded form: prompts (whole, packed, or a piece behind cached context)

A latent row is 512 latent values and 64 key values; expanded heads have 192
query/key channels (128 of their own, 64 shared) and 128 value channels.  All
data are bf16 with fp32 log-sum-exps, lengths and page ids int32, slots and
packed offsets int64.
"""
import math
import random

import torch

own = False

LAT, PE, NOPE, VDIM = 512, 64, 128, 128
ROW = LAT + PE
QK = NOPE + PE
EPS = 1e-6
# Plain values an input page id or a slot holds where nothing was planned.
NO_PAGE = 0


# ---- cases ----

def listed():
    return [
        # a serving step's bookkeeping: every request gets one more token
        dict(name="plan_step", op="plan", requests=256, cached=8192, new=1, page=64, lens=1),
        # admission of a batch of prompts into an empty cache, small pages
        dict(name="plan_prompts", op="plan", requests=64, cached=0, new=4096, page=16, lens=2),
        # the step's new latents into the cache
        dict(name="append_step", op="append", tokens=256, page=64, norm=True),
        # a packed batch of prompts into the cache
        dict(name="append_prompts", op="append", tokens=131072, page=16, norm=True),
        # one user's conversation: latency of a single request
        dict(name="decode_single", op="decode", requests=1, heads=32, new=1, longest=8192, ragged=False, page=64, lens=3),
        # a full serving batch with ragged contexts
        dict(name="decode_batch", op="decode", requests=256, heads=32, new=1, longest=4096, ragged=True, page=64, lens=4),
        # a few long documents, half of the heads, small pages
        dict(name="decode_long", op="decode", requests=8, heads=16, new=1, longest=131072, ragged=True, page=16, lens=5),
        # drafted tokens checked together: three new tokens a request, many heads
        dict(name="decode_drafts", op="decode", requests=48, heads=64, new=3, longest=8192, ragged=True, page=128, lens=6),
        # a short prompt: latency
        dict(name="prefill_short", op="prefill", seqs=1, heads=32, longest=129, context=0, ragged=False, causal=True, lens=7),
        # one long prompt
        dict(name="prefill_prompt", op="prefill", seqs=1, heads=32, longest=8192, context=0, ragged=False, causal=True, lens=8),
        # prompts of many users packed together
        dict(name="prefill_packed", op="prefill", seqs=24, heads=16, longest=2048, context=0, ragged=True, causal=True, lens=9),
        # a piece of a long prompt behind what is cached of it
        dict(name="prefill_piece", op="prefill", seqs=2, heads=16, longest=1024, context=15360, ragged=False, causal=True, lens=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "prefill", "prefill"])
    seed = rng.randrange(1 << 20)
    page = rng.choice([8, 16, 16, 32, 48, 64, 64, 128, 256])
    if op == "plan":
        requests = _log(rng, 1, 1024)
        return dict(op=op, requests=requests, cached=rng.choice([0, _log(rng, 1, 16384)]),
                    new=rng.choice([1, 1, _log(rng, 1, max(1, 131072 // requests))]), page=page, lens=seed)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 131072), page=page, norm=rng.random() < 0.7)
    if op == "decode":
        heads = rng.choice([1, 4, 8, 12, 16, 24, 32, 40, 64, 128])
        new = rng.choice([1, 1, 1, 2, 3, 4])
        requests = _log(rng, 1, 256)
        # padded tokens and score products stay within the largest listed cases'
        most = min(131072, (1 << 20) // requests, 48 * 64 * 3 * 8192 // (requests * heads * new))
        return dict(op=op, requests=requests, heads=heads, new=new, longest=_log(rng, 1, max(1, most)),
                    ragged=rng.random() < 0.6, page=page, lens=seed)
    heads = rng.choice([1, 2, 4, 8, 16, 32])
    seqs = _log(rng, 1, 32)
    pairs = 32 * 8192 * 8192 // 4
    context = rng.choice([0, 0, _log(rng, 1, 8192)])
    longest = _log(rng, 1, 8192)
    while seqs * heads * longest * (longest + context) > pairs:
        longest = max(1, longest // 2)
        context //= 2
    return dict(op=op, seqs=seqs, heads=heads, longest=longest, context=context, ragged=rng.random() < 0.6,
                causal=rng.random() < 0.8, lens=seed)


def _lengths(count, longest, ragged, seed):
    """Lengths that go by the case alone; the first is the longest."""
    rng = random.Random(seed)
    return [longest if (i == 0 or not ragged) else rng.randint(1, longest) for i in range(count)]


def _plan_lengths(case):
    rng = random.Random(case["lens"])
    n = case["requests"]
    cached = [rng.randint(0, case["cached"]) for _ in range(n)]
    return cached, _lengths(n, case["new"], case["new"] > 1, case["lens"] + 1)


def _sequence_lengths(case):
    """Query and key lengths of a prefill case (keys: context and the queries' own)."""
    lq = _lengths(case["seqs"], case["longest"], case["ragged"], case["lens"])
    ctx = _lengths(case["seqs"], case["context"], case["ragged"], case["lens"] + 1) if case["context"] else [0] * case["seqs"]
    return lq, [a + b for a, b in zip(lq, ctx)]


def _pages(tokens, page):
    return -(-tokens // page)


# ---- inputs ----

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(std).to(torch.bfloat16)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    op = case["op"]
    state = {"case": case}
    if op == "plan":
        cached, new = _plan_lengths(case)
        page = case["page"]
        width = max(_pages(c + n, page) for c, n in zip(cached, new)) + 1
        held = [_pages(c, page) for c in cached]
        total = [_pages(c + n, page) for c, n in zip(cached, new)]
        pool = torch.randperm(sum(total) + 64, generator=gen, device=dev).to(torch.int32)
        table = torch.full((len(cached), width), NO_PAGE, dtype=torch.int32, device=dev)
        col = torch.arange(width, device=dev)
        mask = col[None, :] < ints(held)[:, None]
        table[mask] = pool[:sum(held)]
        state.update(cached=ints(cached), new=ints(new), table=table, free=pool[sum(held):].contiguous(), page=page,
                     tokens=sum(new))
    elif op == "append":
        tokens, page = case["tokens"], case["page"]
        pages = _pages(tokens, page) + 1
        rows = normal(tokens, ROW)  # one projection's output: latents and key parts side by side
        slots = torch.randperm(pages * page, generator=gen, device=dev)[:tokens].contiguous()
        weight = torch.rand((LAT,), generator=gen, device=dev) + 0.5
        state.update(c=rows[:, :LAT], k_pe=rows[:, LAT:], slots=slots, cache=normal(pages, page, ROW),
                     weight=weight if case["norm"] else None)
    elif op == "decode":
        n, page = case["requests"], case["page"]
        lens = _lengths(n, case["longest"], case["ragged"], case["lens"])
        held = [_pages(x, page) for x in lens]
        width = max(held)
        pages = sum(held) + 3
        perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.full((n, width), NO_PAGE, dtype=torch.int32, device=dev)
        table[torch.arange(width, device=dev)[None, :] < ints(held)[:, None]] = perm[:sum(held)]
        q = normal(n, case["new"], case["heads"], ROW)
        state.update(q=q, cache=normal(pages, page, ROW), table=table, lens=ints(lens), scale=QK ** -0.5,
                     lse=torch.empty((n, case["new"], case["heads"]), dtype=torch.float32, device=dev))
    else:
        lq, lk = _sequence_lengths(case)
        heads = case["heads"]
        tq, tk = sum(lq), sum(lk)
        kv = normal(1, tk, heads, NOPE + VDIM)  # the up-projection's output: keys and values side by side
        even = not case["ragged"]
        lead = (case["seqs"], -1) if even else (1, -1)
        kv = kv.view(*lead, heads, NOPE + VDIM)
        cu = [torch.tensor([0] + lens, device=dev).cumsum(0) for lens in (lq, lk)]
        q = normal(1, tq, heads, QK).view(*lead, heads, QK)
        state.update(q=q, k=kv[..., :NOPE], v=kv[..., NOPE:], k_pe=normal(1, tk, PE).view(*lead, PE), scale=QK ** -0.5,
                     causal=case["causal"], cu_q=None if even else cu[0], cu_k=None if even else cu[1],
                     most=(max(lq), max(lk)), lse=torch.empty(q.shape[:3], dtype=torch.float32, device=dev))
    return state


# ---- one pass ----

def run(state):
    return {"plan": _run_plan, "append": _run_append, "decode": _run_decode, "prefill": _run_prefill}[state["case"]["op"]](state)


def _run_plan(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_plan
        p = latent_plan(s["cached"], s["new"], s["table"], s["free"], s["page"], s["tokens"])
        return {"table": s["table"], "seq_lens": p["seq_lens"], "cu_seqlens": p["cu_seqlens"], "slot_map": p["slot_map"],
                "pages_taken": p["pages_taken"]}
    page, table = s["page"], s["table"]
    cached, new = s["cached"].long(), s["new"].long()
    total = cached + new
    held = (cached + page - 1) // page
    need = (total + page - 1) // page - held
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)[None, :] - held[:, None]
    taken = (col >= 0) & (col < need[:, None])
    at = (first[:, None] + col).clamp(0, max(0, s["free"].numel() - 1))
    table.copy_(torch.where(taken, s["free"][at], table))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    token = torch.arange(s["tokens"], device=table.device)
    request = torch.searchsorted(cu, token, right=True) - 1
    pos = cached[request] + token - cu[request]
    slots = table[request, pos // page].long() * page + pos % page
    return {"table": table, "seq_lens": total.to(torch.int32), "cu_seqlens": cu, "slot_map": slots,
            "pages_taken": need.sum().to(torch.int32).reshape(1)}


def _run_append(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_append
        return latent_append(s["c"], s["k_pe"], s["slots"], s["cache"], s["weight"], EPS)
    c = s["c"].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    s["cache"].view(-1, ROW)[s["slots"]] = torch.cat([c, s["k_pe"].float()], -1).to(torch.bfloat16)
    return s["cache"]


def _softmax(scores):
    """Probabilities and log-sum-exps of masked (-inf) scores; an empty row gives zeros and -inf."""
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    return p / torch.where(total > 0, total, torch.ones_like(total)), lse.squeeze(-1)


def _run_decode(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_decode
        out = latent_decode(s["q"], s["cache"], s["table"], s["lens"], s["scale"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    q, cache, table, lens = s["q"], s["cache"], s["table"], s["lens"].long()
    n, new, heads, _ = q.shape
    kv = cache[table.long()].reshape(n, -1, ROW).float()
    pos = torch.arange(kv.shape[1], device=q.device)
    kv = torch.where((pos[None, :] < lens[:, None])[..., None], kv, torch.zeros((), device=q.device))
    scores = torch.matmul(q.reshape(n, new * heads, ROW).float(), kv.transpose(1, 2)).mul_(s["scale"])
    seen = lens[:, None] - (new - 1) + torch.arange(new, device=q.device)[None, :]
    mask = pos[None, None, None, :] < seen[:, :, None, None]
    scores = scores.view(n, new, heads, -1).masked_fill(~mask, -math.inf)
    p, lse = _softmax(scores)
    out = torch.matmul(p.view(n, new * heads, -1), kv[..., :LAT])
    s["lse"].copy_(lse)
    return {"out": out.view(n, new, heads, LAT).to(torch.bfloat16), "lse": s["lse"]}


def _run_prefill(s):
    if own:
        from kimi_delta_attention_05_gb300 import latent_prefill
        out = latent_prefill(s["q"], s["k"], s["k_pe"], s["v"], s["scale"], lse=s["lse"], cu_seqlens=s["cu_q"],
                             cu_seqlens_k=s["cu_k"], causal=s["causal"])
        return {"out": out, "lse": s["lse"]}
    q, k, k_pe, v = s["q"], s["k"], s["k_pe"], s["v"]
    heads, dev = q.shape[2], q.device
    if s["cu_q"] is None:
        n = q.shape[0]
        lq = torch.full((n,), q.shape[1], device=dev)
        lk = torch.full((n,), k.shape[1], device=dev)
        at_q = at_k = None
    else:  # packed sequences side by side, each padded to the longest
        cu_q, cu_k = s["cu_q"], s["cu_k"]
        lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
        at_q = (cu_q[:-1, None] + torch.arange(s["most"][0], device=dev)[None, :]).clamp(max=q.shape[1] - 1)
        at_k = (cu_k[:-1, None] + torch.arange(s["most"][1], device=dev)[None, :]).clamp(max=k.shape[1] - 1)
        q, k, k_pe, v = q[0][at_q], k[0][at_k], k_pe[0][at_k], v[0][at_k]
    keys = torch.cat([k.float(), k_pe.float()[:, :, None, :].expand(-1, -1, heads, -1)], -1)
    scores = torch.matmul(q.float().transpose(1, 2), keys.permute(0, 2, 3, 1)).mul_(s["scale"])
    i = torch.arange(scores.shape[2], device=dev)[None, :, None]
    j = torch.arange(scores.shape[3], device=dev)[None, None, :]
    mask = j < lk[:, None, None]
    if s["causal"]:
        mask = mask & (j <= i + (lk - lq)[:, None, None])
    p, lse = _softmax(scores.masked_fill_(~mask[:, None], -math.inf))
    out = torch.matmul(p, v.float().transpose(1, 2)).transpose(1, 2)
    lse = lse.transpose(1, 2)
    if at_q is not None:
        real = torch.arange(q.shape[1], device=dev)[None, :] < lq[:, None]
        out, lse = out[real][None], lse[real][None]
    s["lse"].copy_(lse)
    return {"out": out.to(torch.bfloat16), "lse": s["lse"]}


# ---- what a pass cannot do without ----

def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _plan_lengths(case)
        taken = sum(_pages(c + n, case["page"]) - _pages(c, case["page"]) for c, n in zip(cached, new))
        n = case["requests"]
        # lengths in and out, offsets, taken pages in and out, slots
        return {"bytes": 12 * n + 8 * (n + 1) + 8 * taken + 8 * sum(new), "flops": 0}
    if op == "append":
        return {"bytes": case["tokens"] * (2 * 2 * ROW + 8), "flops": case["tokens"] * (4 * LAT if case["norm"] else 0)}
    if op == "decode":
        n, rows, page = case["requests"], case["heads"] * case["new"], case["page"]
        lens = _lengths(n, case["longest"], case["ragged"], case["lens"])
        moved = 2 * ROW * sum(lens) + 4 * sum(_pages(x, page) for x in lens) + 4 * n
        seen = sum(max(0, x - i) for x in lens for i in range(case["new"])) * case["heads"]
        return {"bytes": moved + n * rows * (2 * ROW + 2 * LAT + 4), "flops": 2 * (ROW + LAT) * seen}
    lq, lk = _sequence_lengths(case)
    heads = case["heads"]
    if case["causal"]:  # query i of a sequence sees the context and the i + 1 first of its own tokens
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
    else:
        pairs = sum(a * b for a, b in zip(lq, lk))
    moved = 2 * sum(lq) * heads * (QK + VDIM) + 4 * sum(lq) * heads + 2 * sum(lk) * (heads * (NOPE + VDIM) + PE)
    return {"bytes": moved, "flops": 2 * (QK + VDIM) * heads * pairs}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":  # whole numbers: no value in 64 bits to be compared with
        return None
    if op == "append":
        cache = s["cache"].double()
        c = s["c"].double()
        if s["weight"] is not None:
            c = s["weight"].double() * c / torch.sqrt((c * c).sum(1, keepdim=True) / LAT + EPS)
        page = s["slots"] // case["page"]
        offset = s["slots"] % case["page"]
        cache[page, offset, :LAT] = c
        cache[page, offset, LAT:] = s["k_pe"].double()
        return cache
    if op == "decode":
        n, new, heads, page = case["requests"], case["new"], case["heads"], case["page"]
        out = torch.zeros((n, new, heads, LAT), dtype=torch.float64, device=s["q"].device)
        lse = torch.full((n, new, heads), -math.inf, dtype=torch.float64, device=s["q"].device)
        lens = _lengths(n, case["longest"], case["ragged"], case["lens"])
        for b, length in enumerate(lens):
            rows = s["cache"][s["table"][b, :_pages(length, page)].long()].reshape(-1, ROW)[:length].double()
            for i in range(new):
                seen = length - (new - 1 - i)
                if seen > 0:
                    x = s["scale"] * (s["q"][b, i].double() @ rows[:seen].T)
                    lse[b, i] = torch.logsumexp(x, 1)
                    out[b, i] = torch.softmax(x, 1) @ rows[:seen, :LAT]
        return {"out": out, "lse": lse}
    lq, lk = _sequence_lengths(case)
    heads = case["heads"]
    q, k, v = (s[x].reshape(-1, heads, s[x].shape[-1]) for x in ("q", "k", "v"))
    k_pe = s["k_pe"].reshape(-1, PE)
    out = torch.zeros((q.shape[0], heads, VDIM), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], heads), -math.inf, dtype=torch.float64, device=q.device)
    a = b = 0
    for nq, nk in zip(lq, lk):
        kp = k_pe[b:b + nk].double()
        for h in range(heads):
            qh = q[a:a + nq, h].double()
            x = (qh[:, :NOPE] @ k[b:b + nk, h].double().T + qh[:, NOPE:] @ kp.T) * s["scale"]
            if case["causal"]:
                x = x + torch.full_like(x, -math.inf).triu_(nk - nq + 1)
            lse[a:a + nq, h] = torch.logsumexp(x, 1)
            out[a:a + nq, h] = torch.softmax(x, 1) @ v[b:b + nk, h].double()
        a, b = a + nq, b + nk
    shape = s["q"].shape
    return {"out": out.view(*shape[:3], VDIM), "lse": lse.view(*shape[:3])}
