"""Pins of oracle/latent.py's page calls: worked by hand, and the counts of holders
against a count over the tables."""
import random

import pytest

from oracle import latent as L


def _holders(cached, table, page, pages):
    n = [0] * pages
    for b, c in enumerate(cached):
        for at in range(-(-c // page)):
            n[table[b][at]] += 1
    return n


def test_fork_by_hand():
    # request 0: 20 tokens in pages 7, 3, 5 of 8; 1 takes all, 2 takes 16, 3 takes 3
    table = [[7, 3, 5, -1], [9, 9, 9, 9], [9, 9, 9, 9], [9, 9, 9, 9]]
    r = L.fork([0, 0, 0], [1, 2, 3], [20, 16, 3], [20, 0, 0, 0], table, [1, 2, 4], [0] * 10, 8)
    assert r["table"] == [[7, 3, 5, -1], [7, 3, 1, 9], [7, 3, 9, 9], [2, 9, 9, 9]]
    assert r["copies"] == [(1, 5, 4), (2, 7, 3)] and r["pages_taken"] == [2] and r["seq_lens"] == [20, 20, 16, 3]
    assert r["shares"] == [0, 0, 0, 2, 0, 0, 0, 2, 0, 0]


def test_release_by_hand():
    # pages 7 and 3 are held by both rows; 0 keeps 9 tokens (two pages), 1 nothing
    table, shares = [[7, 3, 5], [7, 3, 1]], [0, 0, 0, 1, 0, 0, 0, 1]
    r = L.release([1, 0], [0, 9], [20, 18], table, shares, 8)
    assert r == dict(shares=[0] * 8, seq_lens=[9, 0], pages=[1, 5] + [-1] * 6, count=[2])
    assert L.release([0, 1], None, [20, 18], table, shares, 8)["pages"][:4] == [1, 3, 5, 7]


def test_compact_by_hand():
    r = L.compact([20, 17], [[7, 2, 5, 9], [7, 0, 4, 9]], [0, 0, 0, 0, 0, 0, 0, 1, 0, 0], 8)
    # held 0 2 4 5 7: five pages, places 1 and 3 get 5 and 7
    assert r["moves"] == [(1, 5), (3, 7)] and r["pages_used"] == [5]
    assert r["table"] == [[3, 2, 1, 9], [3, 0, 4, 9]] and r["shares"] == [0, 0, 0, 1, 0, 0, 0, 0, 0, 0]
    assert r["page_map"] == [0, -1, 2, -1, 4, 1, -1, 3, -1, -1]


@pytest.mark.parametrize("seed", range(20))
def test_counts_are_those_of_the_tables(seed):
    """After any forks, releases and a compaction: shares = holders - 1, free pages have none, every page is
    either held or free."""
    rng = random.Random(seed)
    page, pages, B, width = 8, 60, 6, 9
    cached, table, shares, free = [0] * B, [[-1] * width for _ in range(B)], [0] * pages, list(range(pages))
    for _ in range(12):
        act = rng.choice(["grow", "fork", "release", "compact"])
        idle = [b for b in range(B) if cached[b] == 0]
        live = [b for b in range(B) if cached[b] > 0]
        if act == "grow" and idle:
            new = [rng.randint(1, 60) if b in idle[:2] else 0 for b in range(B)]
            if sum(-(-n // page) for n in new) <= len(free):
                p = L.plan(cached, new, table, free, page, sum(new))
                cached, table, free = p["seq_lens"], p["table"], free[p["pages_taken"][0]:]
        elif act == "fork" and idle and live and len(free) >= len(idle):
            of = [rng.choice(live) for _ in idle]
            r = L.fork(of, idle, [rng.randint(0, cached[b]) for b in of], cached, table, free, shares, page)
            cached, table, shares, free = r["seq_lens"], r["table"], r["shares"], free[r["pages_taken"][0]:]
        elif act == "release" and live:
            rows = rng.sample(live, rng.randint(1, len(live)))
            r = L.release(rows, [rng.choice([0, rng.randint(0, cached[b])]) for b in rows], cached, table, shares, page)
            cached, shares = r["seq_lens"], r["shares"]
            free = free + r["pages"][:r["count"][0]]
        elif act == "compact":
            r = L.compact(cached, table, shares, page)
            table, shares, free = r["table"], r["shares"], list(range(r["pages_used"][0], pages))
        holders = _holders(cached, table, page, pages)
        assert shares == [max(0, n - 1) for n in holders]
        assert sorted(free + [p for p, n in enumerate(holders) if n]) == list(range(pages))
