"""Latent attention on the GPU against oracle/latent.py (fp64).

Bounds, fixed before the first run.  With spread = sum_j p_j |v_j| and reach =
scale max_j sum_d |q_d k_jd| from the oracle:
  scores: fp32 sums of up to 576 exact products, each addition rounded or cut
          to 24 bits:          ds = 576 2^-23 reach
  out:    weights rounded to bf16 (8 significant bits: 2^-8) and the result too
          (2^-8), weights off by e^ds above and below the fraction, fp32 sums
          over n weights:      |o - ref| <= (2^-7 + 2^-12 + 2 ds + n 2^-24) spread
  lse:    |z - ref| <= ds + n 2^-24 + 2^-20 (1 + |ref|)
Empty rows are exact: zeros and -inf.
"""
import numpy as np
import pytest
import torch

from kimi_delta_attention_05_gb300 import KdaError, get_status, latent as M
from oracle import latent as L

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _rand(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _check(out, lse, ref, n):
    o, z, spread, reach = ref
    ds = 576 * 2.0 ** -23 * reach
    got, gz = _f64(out), _f64(lse)
    assert np.isfinite(got).all()
    tol = (2.0 ** -7 + 2.0 ** -12 + 2 * ds[..., None] + n * 2.0 ** -24) * spread
    worst = np.abs(got - o) - tol
    assert (worst <= 0).all(), f"out beyond its bound by {worst.max():.3e}"
    empty = np.isneginf(z)
    assert (np.isneginf(gz) == empty).all() and (got[empty] == 0).all()
    off = np.abs(gz[~empty] - z[~empty]) - (ds[~empty] + n * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(z[~empty])))
    assert (off <= 0).all(), f"lse beyond its bound by {off.max():.3e}"


@pytest.fixture(autouse=True)
def _clean_status():
    get_status()
    yield


# ---- plan ----

@pytest.mark.parametrize("cached,new,page", [
    ([0], [1], 8), ([7], [1], 8), ([8], [1], 8), ([], [], 64), ([5, 0, 16], [0, 0, 0], 16),
    ([0, 8, 5, 0, 31], [9, 1, 2, 0, 70], 8), ([0, 100], [3000, 1], 48),
])
def test_plan(cached, new, page):
    _plan(cached, new, page, 0)
    _plan(cached, new, page, 5)


def test_plan_many_requests():
    rng = np.random.default_rng(3)
    _plan(rng.integers(0, 300, 3000).tolist(), rng.integers(0, 5, 3000).tolist(), 16, 1)
    _plan([0] * 16384, [1] * 16384, 8, 0)  # the most requests of one call


def _plan(cached, new, page, spare, stride=3):
    rng = np.random.default_rng(1)
    total = [c + n for c, n in zip(cached, new)]
    width = max([-(-t // page) for t in total] + [1])
    held = [-(-c // page) for c in cached]
    need = sum(-(-t // page) for t in total) - sum(held)
    ids = rng.permutation(sum(held) + need + 4)
    rows, at = [], 0
    for h in held:
        rows.append(ids[at:at + h].tolist() + [-7] * (width - h))
        at += h
    free = ids[at:].tolist()
    ref = L.plan(cached, new, rows, free, page, sum(new) + spare)
    i32 = dict(dtype=torch.int32, device="cuda")
    wide = torch.full((len(cached), width + stride), -9, **i32)
    table = wide[:, :width]
    table.copy_(torch.tensor(rows, **i32).reshape(len(cached), width))
    p = M.latent_plan(torch.tensor(cached, **i32), torch.tensor(new, **i32), table, torch.tensor(free, **i32), page,
                      sum(new) + spare)
    assert table.tolist() == ref["table"] and (wide[:, width:] == -9).all()
    for k in ("seq_lens", "cu_seqlens", "slot_map", "pages_taken"):
        assert p[k].tolist() == ref[k], k
    assert get_status() == 0


@pytest.mark.parametrize("cached,new,width,free,tokens,code", [
    ([3, 0], [1, 20], 2, 9, 30, 18),   # 20 tokens need 3 pages, the table has 2
    ([3, 0], [1, 9], 3, 9, 9, 18),     # 10 tokens, 9 slots
    ([3, -1], [1, 9], 3, 9, 30, 18),
    ([3, 0], [1, -9], 3, 9, 30, 18),
    ([3, 0], [1, 2 ** 31 - 1], 3, 9, 30, 18),
    ([3, 0], [8, 9], 3, 2, 30, 19),    # needs 3 pages of 2
])
def test_plan_refuses_on_the_device(cached, new, width, free, tokens, code):
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((2, width), -7, **i32)
    p = M.latent_plan(torch.tensor(cached, **i32), torch.tensor(new, **i32), table, torch.arange(free, **i32), 8, tokens)
    assert get_status() == code and get_status() == 0
    assert (table == -7).all() and p["seq_lens"].tolist() == cached and not p["cu_seqlens"].any()
    assert (p["slot_map"] == -1).all() and p["pages_taken"].tolist() == [0]


# ---- append ----

@pytest.mark.parametrize("T", [0, 1, 7, 300])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("side_by_side", [False, True])
def test_append(T, norm, side_by_side):
    gen = torch.Generator().manual_seed(T + 2)
    rows = _rand(gen, T, 600, std=3.0).cuda()
    c, pe = (rows[:, :512], rows[:, 512:576]) if side_by_side else (rows[:, :512].contiguous(), rows[:, 512:576].contiguous())
    big = _rand(gen, 50, 2, 8, 640).cuda()
    cache = big[:, 1, :, :576]  # one layer of an interleaved cache, padded rows
    before = big.clone()
    slots = torch.randperm(400, generator=gen)[:T].cuda()
    if T > 2:
        slots[1] = -1
    w = (torch.rand(512, generator=gen) + 0.5).cuda() if norm else None
    assert M.latent_append(c, pe, slots, cache, w, 1e-5) is cache
    want = before[:, 1, :, :576].clone()
    ok = slots >= 0
    at = slots[ok]
    got = cache[at // 8, at % 8]
    assert torch.equal(got[:, 512:], pe[ok])
    if norm:  # fp32 arithmetic and one rounding to bf16: 2^-8, with 2^-16 for the fp32 steps
        ref = L.normalised(_f64(c[ok]), _f64(w), 1e-5)
        assert (np.abs(_f64(got[:, :512]) - ref) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + 1e-38).all()
    else:
        assert torch.equal(got[:, :512], c[ok])
    want[at // 8, at % 8] = got
    assert torch.equal(cache, want) and torch.equal(big[:, 0], before[:, 0]) and torch.equal(big[..., 576:], before[..., 576:])
    assert get_status() == 0


def test_append_of_zero_rows_and_slots_outside():
    cache = torch.full((2, 8, 576), 2.0, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")
    M.latent_append(c, c[:, :64], torch.tensor([5, 16, 1 << 40], device="cuda"), cache, torch.ones(512, device="cuda"))
    assert get_status() == 20  # two slots past the 16 of the cache: skipped
    assert (cache.view(16, 576)[5] == 0).all() and cache.sum() == 15 * 576 * 2


# ---- decode ----

def _paged(gen, lens, page, spare=3, behind=NAN, width=None):
    """A shuffled cache whose rows behind the lengths, and pages nobody holds, are `behind`."""
    need = [-(-n // page) for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=gen).tolist()
    cache = torch.full((sum(need) + spare, page, 576), behind, dtype=torch.bfloat16)
    width = max(need + [1]) if width is None else width
    table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)  # never to be followed
    at = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = perm[at]
            cnt = min(page, n - j * page)
            cache[perm[at], :cnt] = _rand(gen, cnt, 576)
            at += 1
    return cache, table


def _decode(lens, R, H, page, seed=0, std=1.0, **kw):
    gen = torch.Generator().manual_seed(seed)
    cache, table = _paged(gen, lens, page)
    q = _rand(gen, len(lens), R, H, 576, std=std)
    lse = torch.full((len(lens), R, H), NAN, device="cuda")
    out = M.latent_decode(q.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 192 ** -0.5,
                          lse=lse, **kw)
    ref = L.absorbed(_f64(q), _f64(cache), table.tolist(), lens, 192 ** -0.5)
    _check(out, lse, ref, max(lens + [1]))
    assert get_status() == 0
    return out, lse


@pytest.mark.parametrize("lens", [[1], [0], [64], [65], [0, 1, 2, 63, 64, 65, 127, 128, 129], [700, 3, 0, 1300]])
@pytest.mark.parametrize("page", [8, 64])
def test_decode_lengths(lens, page):
    _decode(lens, 1, 16, page)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 192, 256])
def test_decode_page_sizes(page):
    _decode([500, 77, 1], 1, 8, page, seed=page)


@pytest.mark.parametrize("H", [1, 3, 16, 17, 32, 40, 64, 65, 128])
@pytest.mark.parametrize("R", [1, 2, 4])
def test_decode_heads_and_new_tokens(H, R):
    """Query rows R * H below, at and past every tile width; lengths below R leave rows empty."""
    _decode([200, 2, 65, 0], R, H, 16, seed=H + R)


def test_decode_long_split_over_the_gpu():
    _decode([20000], 1, 4, 64)
    _decode([9000, 1, 5000], 2, 8, 128)


def test_decode_large_scores():
    """Scores of some hundreds: the running maximum moves many times."""
    _decode([1500, 400], 1, 16, 64, std=30.0)


@pytest.mark.parametrize("step", [1.0, -1.0])
def test_decode_maxima_that_move_with_the_position(step):
    """Every row scores higher (or lower) than the one before, by 0.05 a token over 2000 tokens."""
    n, H = 2000, 8
    cache = torch.zeros(40, 64, 576, dtype=torch.bfloat16)
    cache[..., :512] = _rand(torch.Generator().manual_seed(1), 40, 64, 512)
    cache[..., 512:] = 0
    pos = torch.arange(40 * 64).view(40, 64)
    cache[..., 512] = (step * 0.05 * pos).to(torch.bfloat16)
    q = torch.zeros(1, 1, H, 576, dtype=torch.bfloat16)
    q[..., 512] = torch.linspace(0.25, 2, H).to(torch.bfloat16)
    table = torch.arange(40, dtype=torch.int32)[None]
    lse = torch.empty(1, 1, H, device="cuda")
    out = M.latent_decode(q.cuda(), cache.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 1.0, lse=lse)
    _check(out, lse, L.absorbed(_f64(q), _f64(cache), table.tolist(), [n], 1.0), n)


def test_decode_out_of_range_lengths_and_pages():
    gen = torch.Generator().manual_seed(4)
    cache, table = _paged(gen, [128, 128, 128], 64, behind=0.0)
    table[1, 0] = -3
    table[2, 1] = cache.shape[0]
    q = _rand(gen, 3, 1, 16, 576)
    lse = torch.empty(3, 1, 16, device="cuda")

    def run(lens):
        return M.latent_decode(q.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.07, lse=lse)

    out = run([500, 128, 128])  # 500 is taken as the table's 128; bad pages read as zero rows
    assert get_status() in (18, 20)
    zero = torch.cat([cache, torch.zeros(1, 64, 576, dtype=torch.bfloat16)])
    fixed = table.clone()
    fixed[1, 0] = fixed[2, 1] = cache.shape[0]
    _check(out, lse, L.absorbed(_f64(q), _f64(zero), fixed.tolist(), [128] * 3, 0.07), 128)
    out = run([-5, 0, 0])
    assert get_status() == 18
    assert not out.any() and torch.isneginf(lse).all()


def test_decode_strided_cache_and_table():
    gen = torch.Generator().manual_seed(6)
    lens, page = [150, 33], 16
    cache, table = _paged(gen, lens, page)
    big = torch.full((cache.shape[0], 3, page, 640), NAN, dtype=torch.bfloat16, device="cuda")
    view = big[:, 1, :, :576]
    view.copy_(cache)
    wide = torch.full((2, table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table.cuda()
    q = _rand(gen, 2, 1, 32, 576)
    lse = torch.empty(2, 1, 32, device="cuda")
    out = M.latent_decode(q.cuda(), view, wide[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32).cuda(), 0.07, lse=lse)
    _check(out, lse, L.absorbed(_f64(q), _f64(cache), table.tolist(), lens, 0.07), 150)


def test_decode_cache_past_32_bit_offsets():
    """Pages behind element 2^31 (and byte 2^32) of the cache."""
    pages, page = 120000, 64  # 4.4e9 elements, 8.8 GB
    cache = torch.empty(pages, page, 576, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(8)
    ids = torch.tensor([[pages - 1, 70001, pages - 2, 0]], dtype=torch.int32)
    rows = _rand(gen, 4, page, 576)
    small = rows.clone()
    cache[ids[0].long().cuda()] = rows.cuda()
    slot = torch.tensor([(pages - 1) * page + 5], device="cuda")
    new = _rand(gen, 1, 576)
    M.latent_append(new[:, :512].cuda(), new[:, 512:].cuda(), slot, cache)
    small[0, 5] = new[0]
    q = _rand(gen, 1, 1, 16, 576)
    lse = torch.empty(1, 1, 16, device="cuda")
    out = M.latent_decode(q.cuda(), cache, ids.cuda(), torch.tensor([250], dtype=torch.int32).cuda(), 0.07, lse=lse)
    _check(out, lse, L.absorbed(_f64(q), _f64(small), [[0, 1, 2, 3]], [250], 0.07), 250)


def _decode_state(seed=9, lens=(900, 4000, 37, 0, 2500), H=32, page=64):
    gen = torch.Generator().manual_seed(seed)
    cache, table = _paged(gen, list(lens), page)
    q = _rand(gen, len(lens), 1, H, 576)
    return q.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def test_decode_is_deterministic_whatever_the_workspace_holds():
    q, cache, table, lens = _decode_state()
    need = M.latent_decode_workspace_bytes(*q.shape[:3], cache, table)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda")
        lse = torch.empty(q.shape[:3], device="cuda")
        out = M.latent_decode(q, cache, table, lens, 0.07, lse=lse, workspace=ws)
        if first is None:
            first = out.clone(), lse.clone()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_decode_on_another_stream_and_in_a_graph():
    q, cache, table, lens = _decode_state()
    ref_lse = torch.empty(q.shape[:3], device="cuda")
    ref = M.latent_decode(q, cache, table, lens, 0.07, lse=ref_lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lse = torch.empty_like(ref_lse)
    out = M.latent_decode(q, cache, table, lens, 0.07, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    out = torch.zeros_like(ref)
    ws = torch.empty(max(1, M.latent_decode_workspace_bytes(*q.shape[:3], cache, table)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.latent_decode(q, cache, table, lens, 0.07, out, lse, workspace=ws)
    for n in (torch.tensor([901, 4001, 38, 1, 2501]), torch.tensor([900, 4000, 37, 0, 2500])):
        lens.copy_(torch.minimum(n.to(torch.int32), torch.tensor([900, 4000, 37, 0, 2500], dtype=torch.int32)).cuda())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    lens.copy_(torch.tensor([64, 1, 37, 0, 130], dtype=torch.int32))
    g.replay()
    assert torch.equal(out, M.latent_decode(q, cache, table, lens, 0.07))


# ---- prefill ----

def _prefill(lq, lk, H, causal, packed, seed=0, std=1.0, views=True):
    gen = torch.Generator().manual_seed(seed)
    tq, tk = sum(lq), sum(lk)
    lead = (1,) if packed else (len(lq),)
    q = _rand(gen, *lead, tq // lead[0], H, 192, std=std)
    kv = _rand(gen, *lead, tk // lead[0], H, 256)
    pe = _rand(gen, *lead, tk // lead[0], 64)
    k, v = kv[..., :128], kv[..., 128:]
    cu = [torch.tensor([0] + list(np.cumsum(x)), dtype=torch.int64) for x in (lq, lk)]
    dk, dv = (kv.cuda()[..., :128], kv.cuda()[..., 128:]) if views else (k.contiguous().cuda(), v.contiguous().cuda())
    lse = torch.full(q.shape[:3], NAN, device="cuda")
    out = M.latent_prefill(q.cuda(), dk, pe.cuda(), dv, 192 ** -0.5, lse=lse, causal=causal,
                           cu_seqlens=cu[0].cuda() if packed else None, cu_seqlens_k=cu[1].cuda() if packed else None)
    ref = L.expanded(_f64(q), _f64(k), _f64(pe), _f64(v), 192 ** -0.5, causal, cu[0].tolist() if packed else None,
                     cu[1].tolist() if packed else None)
    _check(out, lse, ref, max(lk + [1]))
    assert get_status() == 0


@pytest.mark.parametrize("n", [1, 2, 64, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_lengths(n, causal):
    _prefill([n], [n], 2, causal, False, seed=n)


@pytest.mark.parametrize("lq,lk", [(1, 300), (100, 357), (130, 385), (300, 1), (300, 170), (5, 640), (257, 513)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_behind_context(lq, lk, causal):
    """Fewer queries than keys (cached context) and more (the first queries see nothing)."""
    _prefill([lq], [lk], 1, causal, False, seed=lq)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_packed(causal):
    lq = [3, 0, 130, 1, 300, 64, 5]
    _prefill(lq, lq, 2, causal, True)
    _prefill(lq, [3, 7, 200, 0, 310, 64, 0], 2, causal, True, seed=1)


def test_prefill_dense_batch_contiguous_and_large_scores():
    _prefill([150] * 3, [150] * 3, 3, True, False, views=False)
    _prefill([150] * 2, [280] * 2, 2, True, False, std=40.0)


@pytest.mark.parametrize("lq,lk", [(1024, 1024), (1100, 1100), (1537, 1537), (1030, 2000), (1280, 700), (1040, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_long(lq, lk, causal):
    """Long enough for the form in which two CTAs share a tile: whole and ragged blocks, keys that
    end inside a tile, context before and fewer keys than queries."""
    _prefill([lq], [lk], 1, causal, False, seed=lq)


def test_prefill_long_packed_and_batched():
    _prefill([1500, 0, 2100, 700], [1500, 0, 2200, 650], 1, True, True, seed=5)
    _prefill([1060] * 2, [1200] * 2, 2, True, False, seed=6, std=20.0)


@pytest.mark.parametrize("lq,lk,heads,causal", [([700, 30, 300, 0, 513, 256], [720, 30, 40, 0, 513, 256], 24, True),
                                                ([300, 30, 300, 0, 256], [300, 30, 40, 0, 513], 32, False),
                                                ([2300, 1900, 2100], [2400, 300, 2100], 6, True)])
def test_prefill_packed_in_many_blocks(lq, lk, heads, causal):
    """More blocks of rows and heads than the GPU has SMs (or pairs of them), so that each works on several in
    turn; some blocks in between see no key."""
    _prefill(lq, lk, heads, causal, True, seed=7)


@pytest.mark.parametrize("lq,lk,heads", [(1, 4096, 1), (130, 5000, 2), (700, 4500, 1), (256, 9000, 3), (1030, 6001, 1),
                                         (1500, 4300, 2), (4500, 4100, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_few_rows_many_keys(lq, lk, heads, causal):
    """Few items with many keys: their key tiles are shared out and the parts joined."""
    _prefill([lq], [lk], heads, causal, False, seed=lq)
    _prefill([lq] * 2, [lk] * 2, heads, causal, False, seed=lk, std=8.0)


@pytest.mark.parametrize("lq,lk,heads", [([1], [4097], 1), ([1, 130, 0, 300], [5000, 4300, 100, 9000], 2),
                                         ([600, 257], [700, 12000], 3), ([2100], [9000], 1), ([1500, 1030], [9000, 400], 2),
                                         ([300, 40], [20, 9000], 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_few_rows_many_keys_packed(lq, lk, heads, causal):
    """The same for packed sequences, whose lengths only the device knows."""
    _prefill(lq, lk, heads, causal, True, seed=sum(lk))


def test_prefill_split_packed_repeats_and_refuses():
    """The parts of a packed split call are the same every time; inconsistent offsets write nothing."""
    gen = torch.Generator().manual_seed(10)
    n, keys = 300, 13000
    q, k, pe, v = (_rand(gen, 1, *x).cuda() for x in ((n, 2, 192), (keys, 2, 128), (keys, 64), (keys, 2, 128)))
    cu = torch.tensor([0, 20, 290, 300], device="cuda")
    cu_k = torch.tensor([0, 5000, 12000, keys], device="cuda")
    need = M.latent_prefill_workspace_bytes(1, n, keys, 2, 3)
    assert need > M.latent_prefill_workspace_bytes(1, n, 1000, 2, 3)
    outs = []
    for fill in (0, 255, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        outs.append(M.latent_prefill(q, k, pe, v, 0.07, cu_seqlens=cu, cu_seqlens_k=cu_k, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    out = torch.full_like(outs[0], 5.0)
    M.latent_prefill(q, k, pe, v, 0.07, out=out, cu_seqlens=cu, cu_seqlens_k=torch.tensor([0, 5000, 4000, keys], device="cuda"))
    assert get_status() == 14 and (out == 5.0).all() and get_status() == 0


def test_prefill_split_workspace():
    """Without a workspace a C call is not split; one that is too small is refused; parts do not depend on what
    the workspace holds."""
    gen = torch.Generator().manual_seed(9)
    q, k, pe, v = (_rand(gen, 1, *x).cuda() for x in ((200, 2, 192), (5000, 2, 128), (5000, 64), (5000, 2, 128)))
    lse = torch.empty(1, 200, 2, device="cuda")
    out = M.latent_prefill(q, k, pe, v, 0.07, lse=lse)
    need = M.latent_prefill_workspace_bytes(1, 200, 5000, 2)
    assert need > 0
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        again = torch.empty_like(lse)
        assert torch.equal(M.latent_prefill(q, k, pe, v, 0.07, lse=again, workspace=ws), out) and torch.equal(again, lse)
    with pytest.raises(M.KdaError):
        M.latent_prefill(q, k, pe, v, 0.07, workspace=ws[: need // 2])
    assert M.latent_prefill_workspace_bytes(1, 200, 1000, 2) == 0 < M.latent_prefill_workspace_bytes(1, 200, 5000, 2, 3)


def test_prefill_without_keys():
    _prefill([40], [0], 2, True, False)


@pytest.mark.parametrize("a,b,n", [(70, 220, 310), (700, 2750, 3450), (900, 4200, 6300)])
def test_prefill_neighbours_do_not_touch(a, b, n):
    """NaN and Inf in the sequence before and after (queries, keys, values) stay there."""
    gen = torch.Generator().manual_seed(3)
    H = 2
    q, kv, pe = (_rand(gen, 1, n, *x).cuda() for x in ((H, 192), (H, 256), (64,)))
    cu = torch.tensor([0, a, b, n], device="cuda")
    lse = torch.empty(1, n, H, device="cuda")
    clean = M.latent_prefill(q, kv[..., :128], pe, kv[..., 128:], 0.07, lse=lse, cu_seqlens=cu)[:, a:b].clone()
    clean_lse = lse[:, a:b].clone()
    for bad in (NAN, float("inf")):
        for t in (q, kv, pe):
            t[:, :a] = bad
            t[:, b:] = bad
        out = M.latent_prefill(q, kv[..., :128], pe, kv[..., 128:], 0.07, lse=lse, cu_seqlens=cu)
        assert torch.equal(out[:, a:b], clean) and torch.equal(lse[:, a:b], clean_lse)
    assert np.isfinite(_f64(clean)).all()


@pytest.mark.parametrize("q_off,k_off", [([0, 50, 40, 100], None), ([0, 50, 90], None), ([10, 50, 100], None),
                                         ([0, 50, 100], [0, 60, 90]), ([0, 50, 100], [0, -1, 100])])
def test_prefill_inconsistent_offsets_write_nothing(q_off, k_off):
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.full((1, 100, 2, 128), 5.0, **z)
    cu = [torch.tensor(x, device="cuda") for x in (q_off, k_off if k_off is not None else q_off)]
    M.latent_prefill(torch.ones(1, 100, 2, 192, **z), torch.ones(1, 100, 2, 128, **z), torch.ones(1, 100, 64, **z),
                     torch.ones(1, 100, 2, 128, **z), 0.07, out, cu_seqlens=cu[0], cu_seqlens_k=cu[1])
    assert get_status() == 14
    assert (out == 5.0).all()


def test_prefill_on_another_stream_and_in_a_graph():
    gen = torch.Generator().manual_seed(12)
    q, k, pe, v = (_rand(gen, 1, 300, *x).cuda() for x in ((4, 192), (4, 128), (64,), (4, 128)))
    cu = torch.tensor([0, 100, 300], device="cuda")
    ref = M.latent_prefill(q, k, pe, v, 0.07, cu_seqlens=cu)
    again = M.latent_prefill(q, k, pe, v, 0.07, cu_seqlens=cu)
    assert torch.equal(ref, again)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = M.latent_prefill(q, k, pe, v, 0.07, cu_seqlens=cu, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    out = torch.zeros_like(ref)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.latent_prefill(q, k, pe, v, 0.07, out, cu_seqlens=cu, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


# ---- refusals of the binding ----

def test_types_shapes_and_strides_are_refused():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i = torch.int32
    q, cache, table, lens = z(2, 2, 4, 576), z(3, 8, 576), z(2, 2, d=i), z(2, d=i)
    M.latent_decode(q, cache, table, lens, 1.0)
    for args in ((q.half(), cache, table, lens), (q[..., :512], cache, table, lens), (q, cache.float(), table, lens),
                 (q, cache[..., :512], table, lens), (q, cache, table.long(), lens), (q, cache, table, lens.long()),
                 (q, cache, table[:1], lens), (q.transpose(1, 2), cache, table, lens), (q, cache, table.t(), lens),
                 (q, cache, table, lens.cpu())):
        with pytest.raises(ValueError):
            M.latent_decode(*args, 1.0)
    with pytest.raises(ValueError):
        M.latent_decode(q, cache, table, lens, 1.0, lse=z(2, 1, 4))
    with pytest.raises(KdaError, match="kda_latent_decode.*16"):
        M.latent_decode(q, cache, table, lens, 0.0)
    with pytest.raises(KdaError, match="17"):
        M.latent_decode(q, z(3, 12, 576), table, lens, 1.0)
    with pytest.raises(KdaError, match="15"):
        M.latent_decode(q, z(3, 8, 580)[..., :576], table, lens, 1.0)
    a = [z(2, 5, 3, 192), z(2, 5, 3, 128), z(2, 5, 64), z(2, 5, 3, 128)]
    M.latent_prefill(*a, 1.0)
    for at, bad in ((0, z(2, 5, 3, 128)), (1, z(2, 5, 2, 128)), (2, z(2, 4, 64)), (3, z(2, 5, 3, 128, d=torch.float32)),
                    (1, z(2, 5, 128, 3).transpose(2, 3)),
                    (0, z(3, 7, 3, 192)[:2, :5])):
        with pytest.raises(ValueError):
            M.latent_prefill(*[bad if n == at else t for n, t in enumerate(a)], 1.0)
    with pytest.raises(ValueError):
        M.latent_prefill(*a, 1.0, cu_seqlens_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(KdaError, match="8"):
        M.latent_prefill(*a, 1.0, cu_seqlens=torch.tensor([0, 5], device="cuda"))
    with pytest.raises(ValueError):
        M.latent_append(z(2, 512), z(2, 64), z(2, d=i), cache)
    with pytest.raises(ValueError):
        M.latent_append(z(2, 512), z(3, 64), z(2, d=torch.int64), cache)
    with pytest.raises(ValueError):
        M.latent_plan(lens, z(3, d=i), table, lens, 8, 4)
    with pytest.raises(KdaError, match="3"):
        M.latent_plan(lens, lens, table, lens, 8, -1)
