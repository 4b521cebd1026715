"""Fork, release, compact and copy of cache pages on the GPU against oracle/latent.py:
whole numbers and copied rows, so everything is equal."""
import random

import pytest
import torch

from kimi_delta_attention_05_gb300 import get_status, latent as M
from kimi_delta_attention_05_gb300 import latent_pages as G
from oracle import latent as L

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def _clean_status():
    get_status()
    yield


def _ints(x):
    return torch.tensor(x, **I32)


def _table(rows, spare=3):
    """A view with rows further apart than they are wide, and the memory around it."""
    width = len(rows[0]) if rows else 0
    wide = torch.full((len(rows), width + spare), -9, **I32)
    view = wide[:, :width]
    if rows and width:
        view.copy_(_ints(rows))
    return view, wide


def _cache(pages, page, seed=0):
    """One layer of an interleaved cache with padded rows, and the memory around it."""
    gen = torch.Generator().manual_seed(seed)
    big = torch.randn((pages, 2, page, 640), generator=gen).to(torch.bfloat16).cuda()
    return big[:, 1, :, :576], big


def _same_around(big, before):
    assert torch.equal(big[:, 0], before[:, 0]) and torch.equal(big[..., 576:], before[..., 576:])


def _batch(rng, B, longest, page, extra=5, idle=0):
    """Lengths, table rows and free pages of B requests of which `idle` hold nothing."""
    cached = [0 if b < idle else rng.randint(0, longest) for b in range(B)]
    rng.shuffle(cached)
    held = [-(-c // page) for c in cached]
    ids = list(range(sum(held) + extra))
    rng.shuffle(ids)
    width, rows, at = max(held + [1]) + 1, [], 0
    for h in held:
        rows.append(ids[at:at + h] + [-7] * (width - h))
        at += h
    return cached, rows, ids[at:], len(ids)


# ---- fork ----

def _fork(parents, children, take, cached, rows, free, shares, page, pages, stream=None):
    ref = L.fork(parents, children, take, cached, rows, free, shares, page)
    table, wide = _table(rows)
    cache, big = _cache(pages, page)
    before, want = big.clone(), cache.clone()
    counts = _ints(shares)
    p = G.latent_fork(_ints(parents), _ints(children), _ints(cached), table, _ints(free), counts, cache,
                      None if take is None else _ints(take), stream=stream)
    torch.cuda.synchronize()
    for to, at, n in ref["copies"]:
        want[to, :n] = want[at, :n]
    assert table.tolist() == ref["table"] and (wide[:, table.shape[1]:] == -9).all()
    assert counts.tolist() == ref["shares"] and torch.equal(cache, want)
    assert p["seq_lens"].tolist() == ref["seq_lens"] and p["pages_taken"].tolist() == ref["pages_taken"]
    _same_around(big, before)
    assert get_status(stream) == 0


@pytest.mark.parametrize("page", [8, 16, 48, 64, 256])
@pytest.mark.parametrize("cached", [0, 1, 7, 8, 63, 64, 65, 256, 700])
def test_fork_one(page, cached):
    rows = [list(range(-(-cached // page))) + [-7], [-7] * (-(-cached // page) + 1)]
    pages = len(rows[0]) + 4
    _fork([0], [1], None, [cached, 0], rows, list(range(pages - 2, pages)), [0] * pages, page, pages)


@pytest.mark.parametrize("seed", range(6))
def test_fork_many(seed):
    rng = random.Random(seed)
    page = [8, 16, 64, 64, 128, 32][seed]
    B, idle = 40, 30
    cached, rows, free, pages = _batch(rng, B, 500, page, extra=40, idle=idle)
    live, to = [b for b in range(B) if cached[b]], [b for b in range(B) if not cached[b]]
    to = rng.sample(to, rng.randint(1, len(to)))
    of = [live[0]] * len(to) if seed == 0 else [rng.choice(live) for _ in to]  # one parent of all
    take = None if seed % 2 else [rng.randint(0, cached[b]) for b in of]
    _fork(of, to, take, cached, rows, free, [rng.randint(0, 3) for _ in range(pages)], page, pages)


def test_fork_on_another_stream_and_of_nothing():
    rng = random.Random(9)
    cached, rows, free, pages = _batch(rng, 6, 300, 16, idle=2)
    live, to = [b for b in range(6) if cached[b]], [b for b in range(6) if not cached[b]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _fork(live[:1], to[:1], None, cached, rows, free, [0] * pages, 16, pages, stream=s)
    _fork([], [], None, cached, rows, free, [0] * pages, 16, pages)
    _fork([], [], [], [], [], [], [0] * 3, 16, 3)


def test_fork_the_most_requests_of_a_call():
    B = 16384
    cached = [9, 24] + [0] * (B - 2)
    rows = [[0, 1, -7], [2, 3, 4]] + [[-7, -7, -7]] * (B - 2)
    pages = B + 3
    _fork([b % 2 for b in range(2, B)], list(range(2, B)), None, cached, rows, list(range(5, pages)), [0] * pages, 8, pages)


@pytest.mark.parametrize("parents,children,take,cached,free,code", [
    ([0], [3], None, [9, 0, 0], 4, 18), ([0], [-1], None, [9, 0, 0], 4, 18), ([3], [1], None, [9, 0, 0], 4, 18),
    ([-1], [1], None, [9, 0, 0], 4, 18), ([0, 0], [1, 1], None, [9, 0, 0], 4, 18), ([0, 1], [1, 2], None, [9, 0, 0], 4, 18),
    ([0], [0], None, [9, 0, 0], 4, 18), ([0], [1], [10], [9, 0, 0], 4, 18), ([0], [1], [-1], [9, 0, 0], 4, 18),
    ([0], [1], None, [25, 0, 0], 4, 18), ([0], [1], None, [-1, 0, 0], 4, 18), ([0, 0], [1, 2], None, [9, 0, 0], 1, 19),
])
def test_fork_refuses_on_the_device(parents, children, take, cached, free, code):
    rows = [[0, 1, 2], [-7, -7, -7], [-7, -7, -7]]
    table, _ = _table(rows)
    cache, big = _cache(9, 8)
    before, counts = big.clone(), torch.zeros(9, **I32)
    p = G.latent_fork(_ints(parents), _ints(children), _ints(cached), table, torch.arange(3, 3 + free, **I32), counts, cache,
                      None if take is None else _ints(take))
    assert get_status() == code and get_status() == 0
    assert table.tolist() == rows and torch.equal(big, before) and not counts.any()
    assert p["seq_lens"].tolist() == cached and p["pages_taken"].tolist() == [0]


def test_fork_of_pages_outside_the_cache():
    """Entered, not counted or copied."""
    cache, big = _cache(6, 8)
    before = big.clone()
    table, _ = _table([[-3, 2, 60], [-7, -7, -7], [-7, -7, -7]])
    counts = torch.zeros(6, **I32)
    p = G.latent_fork(_ints([0, 0]), _ints([1, 2]), _ints([20, 0, 0]), table, _ints([4, 99]), counts, cache, _ints([20, 12]))
    assert get_status() == 20
    assert table.tolist() == [[-3, 2, 60], [-3, 2, 4], [-3, 99, -7]] and counts.tolist() == [0, 0, 1, 0, 0, 0]
    assert torch.equal(big, before) and p["pages_taken"].tolist() == [2]


# ---- release ----

def _release(which, keep, cached, rows, shares, page):
    ref = L.release(which, keep, cached, rows, shares, page)
    table, wide = _table(rows)
    before, counts = wide.clone(), _ints(shares)
    p = G.latent_release(_ints(which), _ints(cached), table, counts, page, None if keep is None else _ints(keep))
    assert torch.equal(wide, before) and counts.tolist() == ref["shares"]
    for k in ("seq_lens", "pages", "count"):
        assert p[k].tolist() == ref[k], k
    assert get_status() == 0


@pytest.mark.parametrize("B,longest,page,pages", [(1, 0, 8, 1), (1, 1, 8, 1), (3, 64, 16, 13), (40, 900, 8, 5000),
                                                  (40, 3000, 64, 40000), (7, 20000, 16, 9000)])
@pytest.mark.parametrize("keep", [False, True])
def test_release(B, longest, page, pages, keep):
    """Families of requests that hold the same first pages."""
    rng = random.Random(B + longest)
    cached = [rng.randint(0, longest) for _ in range(B)]
    width, rows, shares, at = -(-longest // page) + 1, [], [0] * pages, 0
    ids = list(range(pages))
    rng.shuffle(ids)
    for b in range(B):
        held = -(-cached[b] // page)
        common = min(held, -(-cached[b - 1] // page)) * rng.randint(0, 2) // 2 if b else 0
        row = rows[-1][:common] if common else []
        for q in row:
            shares[q] += 1
        rows.append(row + ids[at:at + held - common] + [-7] * (width - held))
        at += held - common
    assert at <= pages
    for n in {0, 1, B // 2, B}:
        which = rng.sample(range(B), n)
        _release(which, [rng.randint(0, cached[b]) for b in which] if keep else None, cached, rows, shares, page)


def test_release_of_no_pages_and_no_requests():
    _release([], None, [], [], [0] * 5, 8)
    _release([0, 1], None, [0, 0], [[-7], [-7]], [], 8)


def test_release_the_most_requests_of_a_call():
    B = 16384
    rows = [[b, B + b // 2] for b in range(B)]
    _release(list(range(B)), None, [16] * B, rows, [0] * B + [1] * (B // 2), 8)


def test_release_lists_a_page_once_whatever_its_count_says():
    table, _ = _table([[2, 2, 4], [2, 4, 2]])
    counts = _ints([0, 0, 1, 0, 0])
    p = G.latent_release(_ints([0, 1]), _ints([24, 24]), table, counts, 8)
    assert p["pages"].tolist() == [2, 4, -1, -1, -1] and p["count"].tolist() == [2] and not counts.any()


@pytest.mark.parametrize("which,keep,cached", [
    ([3], None, [9, 9, 9]), ([-1], None, [9, 9, 9]), ([1, 1], None, [9, 9, 9]), ([1], [10], [9, 9, 9]), ([1], [-1], [9, 9, 9]),
    ([0], None, [-1, 9, 9]), ([0], None, [25, 9, 9]),
])
def test_release_refuses_on_the_device(which, keep, cached):
    table, _ = _table([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    counts = _ints([1, 0, 2, 0, 0, 0, 0, 0, 0])
    p = G.latent_release(_ints(which), _ints(cached), table, counts, 8, None if keep is None else _ints(keep))
    assert get_status() == 18 and get_status() == 0
    assert counts.tolist() == [1, 0, 2, 0, 0, 0, 0, 0, 0] and p["seq_lens"].tolist() == cached
    assert p["count"].tolist() == [0] and (p["pages"] == -1).all()


def test_release_passes_over_pages_outside_the_cache():
    table, _ = _table([[0, -1, 2], [3, 9, 5]])
    counts = torch.zeros(9, **I32)
    p = G.latent_release(_ints([0, 1]), _ints([24, 24]), table, counts, 8)
    assert get_status() == 20
    assert p["pages"].tolist() == [0, 2, 3, 5, -1, -1, -1, -1, -1] and not counts.any()


# ---- compact ----

def _compact(cached, rows, shares, page, in_place, pages):
    ref = L.compact(cached, rows, shares, page)
    table, wide = _table(rows)
    cache, big = _cache(pages, page)
    before, want, counts = big.clone(), cache.clone(), _ints(shares)
    for to, at in ref["moves"]:
        want[to] = want[at]
    out = dict(out_table=table, out_shares=counts) if in_place else {}
    p = G.latent_compact(_ints(cached), table, counts, cache, **out)
    assert p["block_table"].tolist() == ref["table"] and p["shares"].tolist() == ref["shares"]
    assert p["page_map"].tolist() == ref["page_map"] and p["pages_used"].tolist() == ref["pages_used"]
    assert torch.equal(cache, want) and (wide[:, table.shape[1]:] == -9).all()
    if in_place:
        assert p["block_table"] is table and p["shares"] is counts
    else:
        assert table.tolist() == rows and counts.tolist() == shares
    _same_around(big, before)
    assert get_status() == 0


@pytest.mark.parametrize("B,longest,page,extra", [(1, 0, 8, 0), (1, 1, 8, 3), (2, 8, 8, 0), (3, 40, 8, 2), (9, 300, 16, 30),
                                                  (9, 300, 16, 500), (20, 900, 64, 1), (5, 700, 256, 20), (30, 2000, 8, 900),
                                                  (30, 2000, 8, 33000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(B, longest, page, extra, in_place):
    rng = random.Random(B + extra)
    cached, rows, _, pages = _batch(rng, B, longest, page, extra=extra)
    shares = [0] * pages
    for b in range(1, B):  # some hold the pages of the request before
        if rng.random() < 0.5:
            for at in range(min(-(-cached[b] // page), -(-cached[b - 1] // page)) // 2):
                rows[b][at] = rows[b - 1][at]
    for b in range(B):
        for at in range(-(-cached[b] // page)):
            shares[rows[b][at]] += 1
    _compact(cached, rows, [max(0, s - 1) for s in shares], page, in_place, pages)


def test_compact_of_nothing():
    _compact([], [], [0, 0, 0], 8, False, 3)
    cache = torch.zeros((0, 8, 576), dtype=torch.bfloat16, device="cuda")
    p = G.latent_compact(_ints([0]), _ints([[-7]]), torch.zeros(0, **I32), cache)
    assert p["block_table"].tolist() == [[-7]] and p["pages_used"].tolist() == [0] and get_status() == 0


@pytest.mark.parametrize("cached", [[9, -1], [25, 3], [2 ** 31 - 1, 3]])
def test_compact_refuses_on_the_device(cached):
    rows, shares = [[8, 1, 2], [3, 4, 5]], [1, 0, 0, 0, 0, 0, 0, 0, 2]
    table, _ = _table(rows)
    cache, big = _cache(9, 8)
    before = big.clone()
    p = G.latent_compact(_ints(cached), table, _ints(shares), cache)
    assert get_status() == 18 and get_status() == 0
    assert p["block_table"].tolist() == rows and p["shares"].tolist() == shares and torch.equal(big, before)
    assert p["page_map"].tolist() == list(range(9)) and p["pages_used"].tolist() == [9]


def test_compact_leaves_pages_outside_the_cache():
    table, _ = _table([[8, -1, 2], [70, 4, -7]])
    cache, big = _cache(9, 8)
    want = cache.clone()
    p = G.latent_compact(_ints([24, 16]), table, torch.zeros(9, **I32), cache)
    assert get_status() == 20
    want[0], want[1] = want[4].clone(), want[8].clone()
    assert p["block_table"].tolist() == [[1, -1, 2], [70, 0, -7]] and p["pages_used"].tolist() == [3] and torch.equal(cache, want)


# ---- copy ----

@pytest.mark.parametrize("page,n", [(8, 0), (8, 1), (8, 7), (16, 5), (24, 100), (64, 33), (256, 3), (8, 3001)])
def test_copy(page, n):
    gen = torch.Generator().manual_seed(n)
    src, _ = _cache(n + 3, page, 1)
    dst, big = _cache(n + 2, page, 2)
    before, want = big.clone(), dst.clone()
    at, to = torch.randperm(n + 3, generator=gen)[:n].cuda(), torch.randperm(n + 2, generator=gen)[:n].cuda()
    want[to] = src[at]
    assert G.latent_copy(src, at.int(), dst, to.int()) is dst
    assert torch.equal(dst, want)
    _same_around(big, before)
    dense = torch.zeros((n + 2, page, 576), dtype=torch.bfloat16, device="cuda")
    G.latent_copy(src, at.int(), dense, to.int())
    assert torch.equal(dense[to], src[at]) and get_status() == 0


def test_copy_within_a_cache_and_of_pages_outside():
    cache, big = _cache(12, 8)
    want = cache.clone()
    want[3], want[0] = want[7].clone(), want[11].clone()
    G.latent_copy(cache, _ints([7, -1, 11, 12, 5, 5]), cache, _ints([3, 4, 0, 1, -1, 12]))
    assert get_status() == 20 and torch.equal(cache, want)


# ---- together ----

def test_a_captured_step_replayed_with_other_values():
    """Fork, release and compact in one graph, replayed with other numbers, lengths and pages."""
    rng = random.Random(5)
    page, B, pages, width = 8, 10, 400, 40

    def batch(seed):
        r = random.Random(seed)
        cached, rows, free, _ = _batch(r, B, 250, page, extra=0, idle=4)
        rows = [x[:width] + [-7] * (width - len(x)) for x in rows]
        used = {p for b in range(B) for p in rows[b][:-(-cached[b] // page)]}
        free = [p for p in range(pages) if p not in used][:4]
        live, to = [b for b in range(B) if cached[b]], [b for b in range(B) if not cached[b]][:4]
        return cached, rows, free, [r.choice(live) for _ in to], to

    cached, rows, free, of, to = batch(0)
    t = dict(cached=_ints(cached), table=_ints(rows), free=_ints(free), of=_ints(of), to=_ints(to),
             counts=torch.zeros(pages, **I32))
    cache, _ = _cache(pages, page)

    def step():
        f = G.latent_fork(t["of"], t["to"], t["cached"], t["table"], t["free"], t["counts"], cache)
        r = G.latent_release(t["of"][:1], f["seq_lens"], t["table"], t["counts"], page)
        c = G.latent_compact(r["seq_lens"], t["table"], t["counts"], cache, out_table=t["table"], out_shares=t["counts"])
        return f, r, c

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, r, c = step()
    for seed in (1, 2, 3):
        cached, rows, free, of, to = batch(seed)
        for k, v in dict(cached=cached, table=rows, free=free, of=of, to=to).items():
            t[k].copy_(_ints(v))
        t["counts"].zero_()
        want = cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        a = L.fork(of, to, None, cached, rows, free, [0] * pages, page)
        b = L.release(of[:1], None, a["seq_lens"], a["table"], a["shares"], page)
        e = L.compact(b["seq_lens"], a["table"], b["shares"], page)
        for where, src, n in a["copies"]:
            want[where, :n] = want[src, :n]
        for where, src in e["moves"]:
            want[where] = want[src]
        assert f["seq_lens"].tolist() == a["seq_lens"] and r["pages"].tolist() == b["pages"]
        assert t["table"].tolist() == e["table"] and t["counts"].tolist() == e["shares"] and torch.equal(cache, want)
        assert c["page_map"].tolist() == e["page_map"]
    assert rng and get_status() == 0


# ---- what would lose or overwrite pages ----

@pytest.mark.parametrize("held", [1, 8, 24])
def test_fork_over_a_request_that_holds_tokens_is_refused(held):
    """Its pages would be held by nobody and free for nobody: they have to be released first."""
    rows = [[0, 1, 2], [3, 4, 5], [-7, -7, -7]]
    table, _ = _table(rows)
    cache, big = _cache(9, 8)
    before, counts = big.clone(), torch.zeros(9, **I32)
    cached, free = [20, held, 0], torch.arange(6, 9, **I32)
    p = G.latent_fork(_ints([0, 0]), _ints([2, 1]), _ints(cached), table, free, counts, cache)
    assert get_status() == 18 and get_status() == 0
    assert table.tolist() == rows and torch.equal(big, before) and not counts.any()
    assert p["seq_lens"].tolist() == cached and p["pages_taken"].tolist() == [0]
    # released, it is a child like any other
    r = G.latent_release(_ints([1]), _ints(cached), table, counts, 8)
    p = G.latent_fork(_ints([0, 0]), _ints([2, 1]), r["seq_lens"], table, free, counts, cache)
    assert p["seq_lens"].tolist() == [20, 20, 20] and counts.tolist()[:2] == [2, 2] and get_status() == 0


# ---- calls large enough for the forms that only they take ----

@pytest.mark.parametrize("B,width,page", [(300, 200, 8), (40, 1000, 64), (16384, 3, 8)])
@pytest.mark.parametrize("keep", [False, True])
def test_release_of_many_entries(B, width, page, keep):
    """More than 32768 entries: counted by a kernel of its own.  Rows in pairs that hold the same first pages."""
    rng = random.Random(B + keep)
    cached = [rng.randint(0, width * page) for _ in range(B)]
    rows, at = [], 0
    pages = sum(-(-c // page) for c in cached) + 7
    ids, shares = list(range(pages)), [0] * pages
    rng.shuffle(ids)
    for b in range(B):
        held = -(-cached[b] // page)
        common = rng.randint(0, min(held, -(-cached[b - 1] // page))) if b % 2 else 0
        row = rows[-1][:common] if common else []
        for q in row:
            shares[q] += 1
        rows.append(row + ids[at:at + held - common] + [-7] * (width - held))
        at += held - common
    for n in (B, B * 9 // 10):
        assert n * width > 32768
        which = rng.sample(range(B), n)
        _release(which, [rng.randint(0, cached[b]) for b in which] if keep else None, cached, rows, shares, page)


def test_release_of_many_entries_refused_and_outside_the_cache():
    width, B = 400, 100
    table = torch.arange(B * width, **I32).view(B, width)
    counts, lens = torch.zeros(B * width, **I32), torch.full((B,), 8 * width, **I32)
    rows = torch.arange(B, **I32)
    rows[70] = 3  # a row twice
    p = G.latent_release(rows, lens, table, counts, 8)
    assert get_status() == 18 and get_status() == 0 and not counts.any() and p["count"].item() == 0
    assert (p["pages"] == -1).all() and torch.equal(p["seq_lens"], lens)
    rows[70] = 70
    table[99, 5], table[0, 0] = -2, B * width
    p = G.latent_release(rows, lens, table, counts, 8)
    assert get_status() == 20 and not counts.any() and p["count"].item() == B * width - 2
    assert p["pages"][:3].tolist() == [1, 2, 3] and not p["seq_lens"].any()


@pytest.mark.parametrize("pages", [65535, 65537, 131071, 131072, 131073, 262145, 300001])
def test_release_of_caches_that_are_listed_in_rounds(pages):
    """131072 pages a round: pages on both sides of every warp's, CTA's and round's run, few and many."""
    rng = random.Random(pages)
    near = sorted({x + d for x in range(0, pages + 1, 16384) for d in (-33, -1, 0, 1, 31, 32, 1023, 1024) if 0 <= x + d < pages})
    for ids in (near, rng.sample(range(pages), 4000), list(range(pages - 9000, pages))):
        ids = list(ids)
        rng.shuffle(ids)
        rows = [ids[:len(ids) // 2], ids[len(ids) // 2:]]
        width = len(rows[1])
        cached = [8 * len(r) for r in rows]
        shares = [0] * pages
        for q in rng.sample(ids, len(ids) // 3):  # held by others too
            shares[q] = 1
        _release([1, 0], None, cached, [r + [-7] * (width - len(r)) for r in rows], shares, 8)


def test_compact_of_a_cache_of_many_pages():
    """2.8 million pages (26 GB): a bit a page takes more shared memory than a kernel has by default; offsets past 32 bits."""
    page, pages = 8, 2800000
    rng = random.Random(4)
    ids = rng.sample(range(pages), 900) + [pages - 1, pages - 2, 0, 5]
    rng.shuffle(ids)
    rows = [ids[:400], ids[400:]]
    width = max(len(r) for r in rows)
    cached, shares = [8 * len(r) - 3 for r in rows], [0] * pages
    for q in ids[:50]:
        shares[q] = 3
    ref = L.compact(cached, [r + [-7] * (width - len(r)) for r in rows], shares, page)
    cache = torch.empty((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    cache[_ints(ids).long()] = torch.randn((len(ids), page, 576), device="cuda").to(torch.bfloat16)
    want = cache[_ints([src for _, src in ref["moves"]]).long()]
    stay = [q for q in ids if q < len(ids)]
    kept = cache[_ints(stay).long()]
    table = _ints([r + [-7] * (width - len(r)) for r in rows])
    p = G.latent_compact(_ints(cached), table, _ints(shares), cache)
    assert p["block_table"].tolist() == ref["table"] and p["pages_used"].tolist() == ref["pages_used"] == [len(ids)]
    assert p["shares"].tolist() == ref["shares"] and p["page_map"].tolist() == ref["page_map"]
    assert torch.equal(cache[_ints([to for to, _ in ref["moves"]]).long()], want) and torch.equal(cache[_ints(stay).long()], kept)
    assert get_status() == 0


def test_fork_and_copy_past_32_bit_offsets():
    """Pages behind element 2^31 (and byte 2^32) of the cache."""
    page, pages = 64, 120000
    cache = torch.empty((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    some = torch.randn((4, page, 576), device="cuda").to(torch.bfloat16)
    far = [pages - 1, pages - 5, 70000, 3]
    cache[_ints(far).long()] = some
    table = _ints([[far[0], far[1]], [-7, -7], [-7, -7]])
    counts = torch.zeros(pages, **I32)
    p = G.latent_fork(_ints([0, 0]), _ints([1, 2]), _ints([100, 0, 0]), table, _ints([far[2], far[3]]), counts, cache, _ints([100, 30]))
    assert p["pages_taken"].item() == 2 and table.tolist() == [far[:2], [far[0], far[2]], [far[3], -7]]
    assert counts[far[0]] == 1 and int(counts.sum()) == 1
    assert torch.equal(cache[far[2], :36], some[1, :36]) and torch.equal(cache[far[2], 36:], some[2, 36:])
    assert torch.equal(cache[far[3], :30], some[0, :30]) and torch.equal(cache[far[3], 30:], some[3, 30:])
    small = torch.randn((3, page, 576), device="cuda").to(torch.bfloat16)
    before = small.clone()
    G.latent_copy(cache, _ints([far[1], far[0]]), small, _ints([2, 0]))
    assert torch.equal(small[2], some[1]) and torch.equal(small[0], some[0]) and torch.equal(small[1], before[1])
    G.latent_copy(small, _ints([1, 2]), cache, _ints([pages - 2, 60000]))
    assert torch.equal(cache[pages - 2], before[1]) and torch.equal(cache[60000], some[1]) and get_status() == 0


@pytest.mark.parametrize("B", [3, 700])
def test_growth_in_a_page_that_others_hold_is_refused(B):
    """A row cut within a page of others: its next token's slot would lie in their page."""
    page, pages = 8, 3 * B + 9
    rows = [[0, 1, 2, -7], [0, 1, 3, -7], [4, 5, 6, -7]] + [[7 + b, -7, -7, -7] for b in range(B - 3)]
    cached = [20, 24, 24] + [3] * (B - 3)
    shares = [1, 1] + [0] * (pages - 2)
    table, counts, free = _ints(rows), _ints(shares), torch.arange(pages - B, pages, **I32)
    lens, new = _ints(cached), torch.ones(B, **I32)
    for keep, held in ((12, True), (16, False), (9, True), (24, False), (0, False)):
        t, c = table.clone(), counts.clone()
        r = G.latent_release(_ints([1]), lens, t, c, page, _ints([keep]))
        before = t.clone()
        p = M.latent_plan(r["seq_lens"], new, t, free, page, B, shares=c)
        if held:
            assert get_status() == 18 and get_status() == 0
            assert torch.equal(t, before) and torch.equal(p["seq_lens"], r["seq_lens"])
            assert (p["slot_map"] == -1).all() and not p["cu_seqlens"].any() and p["pages_taken"].item() == 0
        else:
            assert get_status() == 0 and torch.equal(p["seq_lens"], r["seq_lens"] + 1)
            plain = M.latent_plan(r["seq_lens"], new, before, free, page, B)
            assert torch.equal(t, before) and all(torch.equal(p[k], plain[k]) for k in p)
        # a request without new tokens may keep such a part, and so may one whose others are gone
        none = new.clone()
        none[1] = 0
        assert M.latent_plan(r["seq_lens"], none, t.clone(), free, page, B, shares=c)["seq_lens"][1] == keep
        assert get_status() == 0
        gone = G.latent_release(_ints([0]), r["seq_lens"], t, c, page)
        p = M.latent_plan(gone["seq_lens"], new, t, free, page, B, shares=c)
        assert get_status() == 0 and torch.equal(p["seq_lens"], gone["seq_lens"] + 1)


def test_plan_with_shares_looks_at_no_page_outside_the_cache():
    table = _ints([[0, 99], [-3, -7], [2, -7]])
    p = M.latent_plan(_ints([12, 3, 8]), _ints([1, 1, 1]), table, _ints([5, 6]), 8, 3, shares=_ints([0, 0, 1, 0, 0, 0, 0]))
    assert get_status() == 0 and p["seq_lens"].tolist() == [13, 4, 9] and p["pages_taken"].item() == 1
    with pytest.raises(ValueError, match="shares"):
        M.latent_plan(_ints([1]), _ints([1]), _ints([[0]]), _ints([1]), 8, 1, shares=torch.zeros(3, dtype=torch.int64, device="cuda"))
