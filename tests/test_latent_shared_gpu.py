"""latent_decode_shared on the GPU against every request's attention over its own rows in
64 bits.

Bounds, fixed before the first run, are those of latent_decode (test_latent_gpu.py): with
spread = sum_j p_j |v_j| and reach = scale max_j sum_d |q_d k_jd|,
  scores: ds = 576 2^-23 reach (fp32 sums of up to 576 exact products)
  out:    weights and result rounded to bf16 (2^-8 each), weights off by e^ds above and
          below the fraction, fp32 sums:  (2^-7 + 2^-12 + 2 ds + n 2^-24) spread.  Joining
          parts multiplies each by 2^(lse_k - lse), whose error (ds, and some 2^-20 of
          the logarithms and exponentials) the terms 2 ds and 2^-12 hold.
  lse:    ds + n 2^-24 + 2^-20 (1 + |ref|)
Rows that see nothing are exact: zeros and -inf.
"""
import pytest
import torch

from kimi_delta_attention_05_gb300 import KdaError, get_status, latent as M
from kimi_delta_attention_05_gb300 import latent_pages as G

pytestmark = pytest.mark.gpu

NAN = float("nan")
I32 = dict(dtype=torch.int32, device="cuda")
SCALE = 192 ** -0.5


@pytest.fixture(autouse=True)
def _clean_status():
    get_status()
    yield


def _rand(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def _wide(B, page, R, H):
    """Pages of a table that the call does not take as latent_decode (KDA_LATENT_SHARED_LEAST)."""
    return (1 << 21) // max(1, B * page * max(16, R * H)) + 1


def _batch(members, prefix, tails, page, R, H, seed=0, std=1.0, spare=2, rows=None, wide=True):
    """q, cache, table, lens, cu, prefix as fork leaves them: whole pages of a prefix in one place, the rest of
    it copied; rows behind the lengths NaN, pages of nobody NaN, entries behind the last page not to be followed."""
    gen = torch.Generator().manual_seed(seed)
    group = [g for g, m in enumerate(members) for _ in range(m)]
    lens = [prefix[g] + t for g, t in zip(group, tails)]
    common = [p // page for p in prefix]
    need = sum(common) + sum(-(-n // page) - common[g] for g, n in zip(group, lens))
    ids = torch.randperm(need + spare, generator=gen).tolist()
    cache = torch.full((need + spare, page, 576), NAN, dtype=torch.bfloat16)
    width = max([-(-n // page) for n in lens] + [1]) + 1
    if wide:
        width = max(width, _wide(len(lens), page, R, H))
    table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
    at, start = 0, []
    first = [rows(p) if rows else _rand(gen, p, 576) for p in prefix]
    for g, c in enumerate(common):
        start.append(at)
        for j in range(c):
            cache[ids[at]] = first[g][j * page:(j + 1) * page]
            at += 1
    for b, (g, n) in enumerate(zip(group, lens)):
        c = common[g]
        table[b, :c] = torch.tensor(ids[start[g]:start[g] + c], dtype=torch.int32)
        own = torch.cat([first[g][c * page:], rows(n - prefix[g]) if rows else _rand(gen, n - prefix[g], 576)])
        for j in range(c, -(-n // page)):
            part = own[(j - c) * page:(j - c + 1) * page]
            table[b, j] = ids[at]
            cache[ids[at], :part.shape[0]] = part
            at += 1
    cu = torch.tensor([0] + members).cumsum(0)
    q = _rand(gen, len(lens), R, H, 576, std=std)
    return [x.cuda() for x in (q, cache, table, torch.tensor(lens, dtype=torch.int32), cu,
                               torch.tensor(prefix, dtype=torch.int32))]


def _reference(q, cache, table, lens, scale):
    B, R, H, _ = q.shape
    page = cache.shape[1]
    out = torch.zeros((B, R, H, 512), dtype=torch.float64, device="cuda")
    spread, lse = torch.zeros_like(out), torch.full((B, R, H), -torch.inf, dtype=torch.float64, device="cuda")
    reach = torch.zeros_like(lse)
    for b, n in enumerate(lens.tolist()):
        rows = cache[table[b, :-(-n // page)].long()].reshape(-1, 576)[:n].double() if n > 0 else cache.new_zeros((0, 576)).double()
        for i in range(R):
            seen = max(0, n - (R - 1 - i))
            if seen == 0:
                continue
            k, x = rows[:seen], q[b, i].double()
            s = scale * (x @ k.T)
            lse[b, i] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[b, i], spread[b, i] = p @ k[:, :512], p @ k[:, :512].abs()
            reach[b, i] = scale * (x.abs() @ k.abs().T).amax(1)
    return out, lse, spread, reach


def _check(out, lse, ref, n):
    o, z, spread, reach = ref
    ds = 576 * 2.0 ** -23 * reach
    got = out.double()
    assert torch.isfinite(got).all()
    worst = (got - o).abs() - (2.0 ** -7 + 2.0 ** -12 + 2 * ds[..., None] + n * 2.0 ** -24) * spread
    assert (worst <= 0).all(), f"out beyond its bound by {worst.max().item():.3e}"
    empty = torch.isneginf(z)
    assert torch.equal(torch.isneginf(lse), empty) and not got[empty].any()
    off = (lse.double() - z).abs()[~empty] - (ds[~empty] + n * 2.0 ** -24 + 2.0 ** -20 * (1 + z[~empty].abs()))
    assert (off <= 0).all(), f"lse beyond its bound by {off.max().item():.3e}"


def _run(batch, status=0, scale=SCALE, **kw):
    q, cache, table, lens, cu, prefix = batch
    lse = torch.full(q.shape[:3], NAN, device="cuda")
    out = M.latent_decode_shared(q, cache, table, lens, cu, prefix, scale, lse=lse, **kw)
    _check(out, lse, _reference(q, cache, table, lens.clamp(0, table.shape[1] * cache.shape[1]), scale), max(lens.tolist() + [1]))
    assert get_status() == status
    return out, lse


@pytest.mark.parametrize("page", [8, 16, 48, 64, 256])
@pytest.mark.parametrize("prefix", [0, 1, 64, 127, 128, 129, 255, 256, 383, 640, 1000])
def test_prefix_lengths(prefix, page):
    _run(_batch([5], [prefix], [1, 64, 7, 200, 65], page, 1, 16, seed=prefix + page))


def test_tables_that_hold_little():
    """Taken as latent_decode, whose results they are; groups that do not fit do not show."""
    for H, members, tails in ((16, [3, 2], [5, 64, 1, 2, 70]), (32, [20, 2], [1 + b for b in range(22)]), (128, [2, 2], [5, 64, 1, 2])):
        batch = _batch(members, [300, 129], tails, 16, 1, H, seed=H, wide=False)
        q, cache, table, lens, cu, prefix = batch
        out, lse = _run(batch)
        alone = torch.empty_like(lse)
        assert torch.equal(out, M.latent_decode(q, cache, table, lens, SCALE, lse=alone)) and torch.equal(lse, alone)
        batch[4] = torch.tensor([0, 9, 2], device="cuda")
        assert torch.equal(_run(batch)[0], out)


@pytest.mark.parametrize("more", [-1, 0, 1])
def test_tables_about_as_wide_as_the_limit(more):
    batch = _batch([4, 4], [1000, 600], [20] * 8, 16, 1, 40, seed=30 + more)
    q, cache, table, lens, cu, prefix = batch
    width = (1 << 21) // (8 * 16 * 40) + more
    batch[2] = torch.cat([table, torch.full((8, 9), 1 << 30, **I32)], 1)[:, :width]
    _run(batch)


def _others(batch, broken):
    """Runs a batch in which a request's rows are not finite; checks the other requests."""
    q, cache, table, lens, cu, prefix = batch
    keep = [b for b in range(len(lens)) if b != broken]
    lse = torch.full(q.shape[:3], NAN, device="cuda")
    out = M.latent_decode_shared(q, cache, table, lens, cu, prefix, SCALE, lse=lse)
    _check(out[keep], lse[keep], _reference(q[keep], cache, table[keep], lens[keep], SCALE), max(lens.tolist()))
    assert get_status() == 0
    return out, lse


@pytest.mark.parametrize("value", [NAN, torch.inf, -torch.inf])
@pytest.mark.parametrize("members,H,prefix,own", [([5], 16, 700, 300), ([24, 3], 32, 400, 100), ([9], 64, 128, 700),
                                                  ([3], 16, 9000, 200), ([3, 40], 3, 300, 150)])
def test_rows_that_are_not_finite_stay_with_their_request(members, H, prefix, own, value):
    """Whole items and cut ones; a row near the start, the middle or the end of the broken request."""
    n = sum(members)
    for broken, at in ((0, 0), (1, own // 2), (2, own)):
        batch = _batch(members, [prefix] * len(members), [1 + own + 7 * b % 60 for b in range(n)], 16, 1, H, seed=n + broken)
        q, cache, table, lens = batch[:4]
        at += prefix // 16 * 16 + 16  # (in a page of its own)
        cache[table[broken, at // 16].long(), at % 16, 5] = value
        out, lse = _others(batch, broken)
        if value != value:  # (a row behind the length is never used)
            seen = at < int(lens[broken])
            assert (torch.isnan(out[broken]) == seen).all() and (torch.isnan(lse[broken]) == seen).all()


def test_prefix_rows_that_are_not_finite_and_not_seen():
    """A request that ends before the broken row of the prefix, and one without a token."""
    batch = _batch([6], [600], [30] * 6, 16, 1, 32, seed=9)
    q, cache, table, lens = batch[:4]
    lens[2], lens[4] = 300, 0
    cache[table[0, 400 // 16].long(), 400 % 16, 100] = NAN
    lse = torch.empty(q.shape[:3], device="cuda")
    out = M.latent_decode_shared(*batch, SCALE, lse=lse)
    some = [2, 4]
    _check(out[some], lse[some], _reference(q[some], cache, table[some], lens[some], SCALE), 300)
    assert torch.isnan(out[[0, 1, 3, 5]]).all() and get_status() == 0


@pytest.mark.parametrize("R", [2, 4])
def test_new_rows_that_are_not_finite_and_not_seen_yet(R):
    """The last new token's row is not finite: the ones before it do not see it."""
    batch = _batch([7], [300], [40 + 50 * b for b in range(7)], 16, R, 24, seed=R)
    q, cache, table, lens = batch[:4]
    at = int(lens[3]) - 1
    cache[table[3, at // 16].long(), at % 16] = NAN
    lse = torch.empty(q.shape[:3], device="cuda")
    out = M.latent_decode_shared(*batch, SCALE, lse=lse)
    ref = [x[:, :-1] for x in _reference(q, cache, table, lens, SCALE)]
    _check(out[:, :-1], lse[:, :-1], ref, int(lens.max()))
    assert torch.isnan(out[3, -1]).all() and get_status() == 0


@pytest.mark.parametrize("n", [12, 13])
def test_rows_about_as_many_as_the_limit(n):
    """480 and 520 rows of 40 heads, in tables that hold little."""
    _run(_batch([n], [300], [3 + b for b in range(n)], 16, 1, 40, seed=n, wide=False))


@pytest.mark.parametrize("members", [[1], [2], [1, 1, 1], [1, 5, 0, 3], [0, 0, 4], [9, 0], [2, 17, 1, 30]])
def test_groups(members):
    n = sum(members)
    prefix = [(517 * (g + 1)) % 900 for g in range(len(members))]
    _run(_batch(members, prefix, [1 + 37 * b % 150 for b in range(n)], 16, 1, 8, seed=n))


@pytest.mark.parametrize("H", [1, 3, 16, 17, 32, 40, 64, 65, 128])
@pytest.mark.parametrize("R", [1, 2, 4])
def test_heads_and_new_tokens(H, R):
    """Rows of a group below, at and past a block of 128; requests that begin anywhere in one."""
    _run(_batch([5, 2, 3], [300, 700, 129], [R + 11 * b % 90 for b in range(10)], 16, R, H, seed=H + R))


def test_requests_that_do_not_see_the_whole_prefix():
    """Shorter and empty ones, whose tables are not to be followed, among the others, and first of a group."""
    batch = _batch([4, 5, 3], [600, 400, 300], [40] * 12, 16, 2, 16, seed=3)
    q, cache, table, lens, cu, prefix = batch
    for b, n in ((0, 0), (2, 513), (4, 0), (5, 1), (6, 399), (8, 0), (9, 0), (10, 0)):
        lens[b] = n
        table[b, -(-n // 16):] = 1 << 30
    _run(batch)
    lens.zero_()
    table.fill_(1 << 30)
    out, lse = _run(batch)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("R", [1, 3])
def test_requests_that_end_with_the_prefix(R):
    """No token of their own (R = 1: the prefix's last is the newest); with R = 3 the first ones do not see all of it."""
    for prefix in (256, 300):
        batch = _batch([3, 3], [prefix, prefix], [0, 1, 2, 0, 0, 5], 8, R, 16, seed=prefix)
        _run(batch)


def test_one_long_prefix_split_over_the_gpu():
    _run(_batch([3], [20000], [1, 700, 64], 64, 1, 16, seed=4))
    _run(_batch([2, 2], [9000, 12345], [5000, 1, 64, 100], 128, 2, 8, seed=5))


def test_many_rows():
    """More blocks of rows than there are SMs; tails that are split too."""
    _run(_batch([40, 37, 1], [1500, 700, 300], [10 + 13 * b % 300 for b in range(77)] + [3000], 64, 3, 64, seed=6))


def test_many_groups():
    members = [1 + g % 3 for g in range(300)]
    n = sum(members)
    _run(_batch(members, [(g * 37) % 400 for g in range(300)], [1 + b % 40 for b in range(n)], 16, 1, 16, seed=7))


def test_more_items_than_a_share_keeps_at_hand():
    """Groups of one, each an item of its own: some tens of items a share, some without a token."""
    n = 6000
    lens = [(b * 7) % 5 for b in range(n)]
    _run(_batch([1] * n, [0] * n, lens, 8, 1, 2, seed=31))


def test_the_most_groups_of_a_call():
    """16384 of them, most without requests."""
    members = [0] * 16384
    for g in range(0, 16384, 500):
        members[g] = 1 + g % 3
    members[-1] = 2
    n = sum(members)
    _run(_batch(members, [(g % 400) if m else 0 for g, m in enumerate(members)], [1 + b % 30 for b in range(n)], 16, 1, 16, seed=32))


@pytest.mark.parametrize("H,R", [(1, 1), (3, 2), (200, 1), (65, 3)])
def test_many_requests_an_item_and_many_items_a_request(H, R):
    _run(_batch([150, 40], [260, 129], [R + 29 * b % 300 for b in range(190)], 32, R, H, seed=H))


@pytest.mark.parametrize("long", [0, 700, 6000])
@pytest.mark.parametrize("prefix", [127, 128, 1300, 5000])
def test_groups_of_many_items(prefix, long):
    """Every second item of such a group takes its own tokens first: items that are a share each, and cut ones; a
    request that is far longer than the others, one that does not see the whole prefix, one without a token."""
    tails = [1 + 53 * b % 400 for b in range(25)]
    tails[6] += long
    batch = _batch([25], [prefix], tails, 16, 1, 32, seed=prefix + long)
    batch[3][13], batch[3][14] = 100, 0
    _run(batch)


def test_large_scores():
    _run(_batch([6], [1500], [400, 1, 30, 64, 65, 2], 64, 1, 16, seed=8, std=30.0))


@pytest.mark.parametrize("step", [1.0, -1.0])
def test_maxima_that_move_with_the_position(step):
    """Every row scores higher (or lower) than the one before, by 0.05 a token."""
    batch = _batch([4], [2000], [60, 1, 10, 200], 64, 1, 8, seed=9)
    q, cache, table, lens, cu, prefix = batch
    for b, n in enumerate(lens.tolist()):
        pos = torch.arange(n, device="cuda")
        where = table[b, pos // 64].long()
        cache[where, pos % 64, 512:] = 0
        cache[where, pos % 64, 512] = (step * 0.05 * pos).to(torch.bfloat16)
    q.zero_()
    q[..., 512] = torch.linspace(0.25, 2, 8).to(torch.bfloat16)
    _run(batch, scale=1.0)


def test_groups_and_prefixes_that_do_not_fit():
    """Every request on its own, or the prefix cut to the table; results stay right."""
    for cu in ([0, 3, 2, 6], [1, 3, 5, 6], [0, 2, 4, 5], [0, 2, 4, 7], [0, -1, 4, 6], [0, 2 ** 40, 4, 6]):
        batch = _batch([2, 2, 2], [300, 400, 500], [5] * 6, 16, 1, 16, seed=10)
        batch[4] = torch.tensor(cu, device="cuda")
        _run(batch, status=14)
    for prefix in ([-1, 400, 500], [300, 2 ** 31 - 1, 500]):
        batch = _batch([2, 2, 2], [300, 400, 500], [5] * 6, 16, 1, 16, seed=10)
        batch[5] = torch.tensor(prefix, **I32)
        _run(batch, status=18)


def test_pages_outside_the_cache_read_as_zeros():
    batch = _batch([3], [512], [20] * 3, 64, 1, 16, seed=11)
    q, cache, table, lens, cu, prefix = batch
    table[:, 2], table[:, 5] = -3, cache.shape[0]
    lse = torch.empty(q.shape[:3], device="cuda")
    out = M.latent_decode_shared(q, cache, table, lens, cu, prefix, SCALE, lse=lse)
    assert get_status() == 20
    zero = torch.cat([cache, torch.zeros_like(cache[:1])])
    fixed = table.clone()
    fixed[:, 2] = fixed[:, 5] = cache.shape[0]
    _check(out, lse, _reference(q, zero, fixed, lens, SCALE), 532)


def test_lengths_past_the_table():
    """Taken as the table's; with R = 3 its last tokens are then not seen by the first of the new ones."""
    gen = torch.Generator().manual_seed(12)
    page, width, R = 64, 600, 3
    cache = _rand(gen, 40, page, 576).cuda()
    table = torch.randint(0, 40, (4, width), generator=gen, dtype=torch.int32).cuda()
    table[1], table[2] = table[0], table[0]
    q = _rand(gen, 4, R, 16, 576).cuda()
    cap = page * width
    lens = torch.tensor([10 ** 6, cap, cap + 1, -4], **I32)
    for prefix in (cap, cap - 2, cap - 128, 256):
        _run([q, cache, table, lens, torch.tensor([0, 3, 4], device="cuda"), torch.tensor([prefix, 64], **I32)], status=18)


def test_no_requests_and_refusals():
    batch = _batch([2], [300], [5, 6], 16, 1, 16, seed=13)
    q, cache, table, lens, cu, prefix = batch
    out = M.latent_decode_shared(q[:0], cache, table[:0], lens[:0], cu[:1], prefix[:0], SCALE)
    assert out.shape == (0, 1, 16, 512)
    with pytest.raises(KdaError):
        M.latent_decode_shared(q, cache, table, lens, cu[:1], prefix[:0], SCALE)  # requests without a group
    with pytest.raises(ValueError, match="cu_groups"):
        M.latent_decode_shared(q, cache, table, lens, cu[:1], prefix, SCALE)
    with pytest.raises(ValueError, match="cu_groups"):
        M.latent_decode_shared(q, cache, table, lens, cu.int(), prefix, SCALE)
    with pytest.raises(ValueError, match="prefix_lens"):
        M.latent_decode_shared(q, cache, table, lens, cu, prefix.long(), SCALE)
    with pytest.raises(ValueError, match="prefix_lens"):
        M.latent_decode_shared(q, cache, table, lens, cu, prefix[0], SCALE)
    with pytest.raises(KdaError):
        M.latent_decode_shared(q, cache, table, lens, cu, prefix, -1.0)
    need = M.latent_decode_shared_workspace_bytes(*q.shape[:3], 1, cache, table)
    for ws in (torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(KdaError):
            M.latent_decode_shared(q, cache, table, lens, cu, prefix, SCALE, workspace=ws)
    assert get_status() == 0


def test_strided_cache_and_table():
    batch = _batch([3, 2], [500, 300], [30] * 5, 16, 1, 32, seed=14)
    big = torch.full((batch[1].shape[0], 3, 16, 640), NAN, dtype=torch.bfloat16, device="cuda")
    big[:, 1, :, :576] = batch[1]
    rows = torch.full((5, batch[2].shape[1] + 5), 1 << 30, **I32)
    rows[:, :batch[2].shape[1]] = batch[2]
    batch[1], batch[2] = big[:, 1, :, :576], rows[:, :batch[2].shape[1]]
    _run(batch)


def test_cache_past_32_bit_offsets():
    """Prefix pages behind element 2^31 (and byte 2^32) of the cache."""
    page, pages = 64, 120000
    batch = _batch([3], [300], [20] * 3, page, 1, 16, seed=15)
    small, table = batch[1], batch[2]
    cache = torch.zeros(pages, page, 576, dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([pages - 1 - 7 * i for i in range(small.shape[0])], device="cuda")
    cache[far] = small
    batch[1] = cache
    batch[2] = torch.where(table < small.shape[0], far[table.clamp(max=small.shape[0] - 1).long()].int(), table)
    _run(batch)


def test_deterministic_whatever_the_workspace_holds():
    for batch in (_batch([30, 2], [3000, 1000], [60 + b for b in range(32)], 64, 1, 32, seed=16),
                  _batch([1, 1, 3], [0, 500, 2500], [3000, 1, 2, 500, 40], 16, 2, 8, seed=17)):
        q, cache, table = batch[:3]
        need = M.latent_decode_shared_workspace_bytes(*q.shape[:3], batch[5].shape[0], cache, table)
        first = None
        for fill in (0, 255, 127):
            ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda")
            got = _run(batch, workspace=ws)
            if first is None:
                first = got
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_calls_of_other_sizes_in_turn():
    """Shares of no, one and many items, each call after one that left other items in shared memory and workspace."""
    batches = [_batch([5, 2, 3], [300, 700, 129], [4 + 11 * b % 90 for b in range(10)], 16, 4, 64, seed=40),
               _batch([1] * 3000, [0] * 3000, [(b * 7) % 5 for b in range(3000)], 8, 1, 2, seed=41),
               _batch([3], [9000], [5, 6, 700], 64, 1, 16, seed=42), _batch([2, 9], [128, 0], [1] * 11, 8, 1, 128, seed=43)]
    need = max(M.latent_decode_shared_workspace_bytes(*x[0].shape[:3], x[5].shape[0], x[1], x[2]) for x in batches)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = [_run(x, workspace=ws) for x in batches]
    for k in range(200):
        i = (k * k + k // 3) % len(batches)
        lse = torch.empty_like(want[i][1])
        out = M.latent_decode_shared(*batches[i], SCALE, lse=lse, workspace=ws)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    assert get_status() == 0


def test_on_another_stream_and_in_a_graph():
    batch = _batch([6, 1, 9], [700, 100, 1300], [30 + 5 * b for b in range(16)], 16, 1, 16, seed=18)
    q, cache, table, lens, cu, prefix = batch
    ref, ref_lse = _run(batch)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lse = torch.empty_like(ref_lse)
    out = M.latent_decode_shared(q, cache, table, lens, cu, prefix, SCALE, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and get_status(s) == 0
    out = torch.zeros_like(ref)
    need = M.latent_decode_shared_workspace_bytes(*q.shape[:3], 3, cache, table)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.latent_decode_shared(q, cache, table, lens, cu, prefix, SCALE, out, lse, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    # other queries, groups, prefixes and lengths
    for members, pre, cut in (([6, 10, 0], [256, 129, 5], 3), ([1, 1, 14], [0, 300, 100], 0), ([16, 0, 0], [130, 0, 0], 20)):
        cu.copy_(torch.tensor([0] + members).cumsum(0))
        new = _batch([m for m in members], pre, [40 + b for b in range(16)], 16, 1, 16, seed=cut)
        w = min(table.shape[1], new[2].shape[1])
        table[:, :w] = new[2][:, :w]
        cache[:] = NAN
        n = min(cache.shape[0], new[1].shape[0])
        assert n == new[1].shape[0] and w == new[2].shape[1]
        cache[:n] = new[1]
        q.copy_(new[0])
        lens.copy_(new[3])
        prefix.copy_(new[5])
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, _reference(q, cache, table, lens, SCALE), 2000)
        again, again_lse = _run(batch)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_two_calls_at_once_on_two_streams():
    a = _batch([8, 8], [2000, 1000], [64] * 16, 64, 1, 32, seed=20)
    b = _batch([3, 1], [700, 300], [50] * 4, 16, 2, 16, seed=21)
    want = [_run(x) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for x, s in zip((a, b), streams):
            got.append(M.latent_decode_shared(*x[:6], SCALE, stream=s))
    torch.cuda.synchronize()
    for k, out in enumerate(got):
        assert torch.equal(out, want[k % 2][0])
    assert all(get_status(s) == 0 for s in streams)


def test_samples_of_prompts_from_prompt_to_release():
    """The calls as a server makes them: prompts planned and appended, samples forked from
    them, tokens appended and decoded behind the shared prefixes, samples dropped, the cache compacted, decoded again."""
    gen = torch.Generator().manual_seed(22)
    page, prompts, each, heads = 16, 3, 4, 16
    lens0 = [333, 64, 100]
    B, pages = prompts * (each + 1), 200
    cache = torch.full((pages, page, 576), NAN, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, _wide(B, page, 1, heads)), 1 << 30, **I32)
    shares, free = torch.zeros(pages, **I32), torch.randperm(pages, generator=gen).int().cuda()
    first = [p * (each + 1) for p in range(prompts)]  # a prompt's row, then its samples
    lens = torch.zeros(B, **I32)
    text = {b: torch.zeros((0, 576), dtype=torch.bfloat16) for b in range(B)}  # what each request's rows have to be

    def add(new):
        nonlocal lens, free
        p = M.latent_plan(lens, torch.tensor(new, **I32), table, free, page, sum(new))
        rows = _rand(gen, sum(new), 576)
        M.latent_append(rows[:, :512].cuda(), rows[:, 512:].cuda(), p["slot_map"], cache)
        lens, free = p["seq_lens"], free[int(p["pages_taken"]):]
        for b, x in enumerate(torch.split(rows, new)):
            text[b] = torch.cat([text[b], x])

    def decode(members, prefix):
        q = _rand(gen, B, 1, heads, 576).cuda()
        lse = torch.empty((B, 1, heads), device="cuda")
        cu = torch.tensor([0] + members).cumsum(0).cuda()
        out = M.latent_decode_shared(q, cache, table, lens, cu, torch.tensor(prefix, **I32), SCALE, lse=lse)
        rows = torch.zeros((B, 640, 576), dtype=torch.bfloat16)  # the texts, not the cache
        for b, x in text.items():
            rows[b, :x.shape[0]] = x
        _check(out, lse, _reference(q, rows.cuda(), torch.arange(B, **I32)[:, None], lens, SCALE), 640)

    add([lens0[first.index(b)] if b in first else 0 for b in range(B)])
    parents = [p for p in first for _ in range(each)]
    children = [p + 1 + i for p in first for i in range(each)]
    f = G.latent_fork(torch.tensor(parents, **I32), torch.tensor(children, **I32), lens, table, free, shares, cache)
    lens, free = f["seq_lens"], free[int(f["pages_taken"]):]
    for p, c in zip(parents, children):
        text[c] = text[p]
    for step in range(20):
        add([1] * B)
        if step % 6 == 0:
            decode([each + 1] * prompts, lens0)
    gone = [first[1], first[0] + 1, first[2] + 3, first[2] + 4]
    keep = [0, 0, 110, 48]  # to its own tokens, and to whole pages of the prefix
    r = G.latent_release(torch.tensor(gone, **I32), lens, table, shares, page, torch.tensor(keep, **I32))
    lens, free = r["seq_lens"], torch.cat([free, r["pages"][:int(r["count"])]])
    for b, k in zip(gone, keep):
        text[b] = text[b][:k]
    assert len(set(free.tolist())) == free.numel()
    decode([each + 1] * prompts, lens0)
    c = G.latent_compact(lens, table, shares, cache, out_table=table, out_shares=shares)
    used = int(c["pages_used"])
    assert used + free.numel() == pages
    free = torch.arange(used, pages, **I32)
    cache[used:] = NAN
    decode([each + 1] * prompts, lens0)
    add([2] * B)
    decode([each + 1] * prompts, lens0)
    other = torch.full((pages + 5, page, 576), NAN, dtype=torch.bfloat16, device="cuda")
    held = torch.arange(pages, **I32)
    G.latent_copy(cache, held, other, held + 5)
    table += 5
    cache = other
    decode([each + 1] * prompts, lens0)
    left = G.latent_release(torch.arange(B, **I32), lens, table - 5, shares, page)
    assert int(left["count"]) + free.numel() == pages and not shares.any() and get_status() == 0


def test_both_ctas_of_a_pair_hand_over_what_they_wrote():
    """Weights and cleared rows lie in the shared memory of both CTAs of a pair and are read by products that one of them
    issues: rows on both, many ends of requests (NaN behind them), maxima that move, calls on two streams at once.
    Weights of the tile before, or rows that are not cleared yet, would give other bits in one call of many."""
    a = _batch([30, 2], [1000, 300], [1 + 37 * b % 300 for b in range(32)], 16, 1, 32, seed=50, std=4.0)
    b = _batch([9] * 8, [640] * 8, [3 + 29 * b % 200 for b in range(72)], 8, 3, 16, seed=51, std=4.0)
    want = [_run(x) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    bad = torch.zeros(2, dtype=torch.int64, device="cuda")
    for _ in range(300):
        for k, (x, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                lse = torch.empty_like(want[k][1])
                out = M.latent_decode_shared(*x, SCALE, lse=lse)
                bad[k] += (out != want[k][0]).sum() + (lse != want[k][1]).sum()
    torch.cuda.synchronize()
    assert not bad.any() and all(get_status(s) == 0 for s in streams)


@pytest.mark.parametrize("R,H", [(5, 16), (9, 3), (33, 8), (130, 2), (300, 1)])
def test_many_new_tokens(R, H):
    """A request's rows fill several items, or its new tokens several tiles; requests that have fewer tokens than are new
    (the first ones see none) or do not all see the prefix; the last group is behind a prefix that is longer than R."""
    for prefix in ([0, 200], [128, 1000], [300, R]):
        tails = [R, 1, R + 100, 2, 64, R + 3]
        batch = _batch([3, 3], prefix, tails, 16, R, H, seed=R + H + prefix[1])
        batch[3][1] = min(int(batch[3][1]), R // 2)
        batch[3][5] = 0
        _run(batch)
