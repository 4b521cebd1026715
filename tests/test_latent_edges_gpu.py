"""Latent attention on the GPU at the edges of what its interface accepts:
buffers at the smallest alignment, and the forms that large calls take."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_05_gb300 import KdaError, get_status, latent as M
from oracle import latent as L
from tests.test_latent_gpu import NAN, _check, _decode, _f64, _paged, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    get_status()
    yield


# ---- prefill: an `out` on a 16-byte boundary that is not one of 32 ----

@pytest.mark.parametrize("lq,lk,heads,packed", [
    ([300], [300], 3, False),                       # single CTAs
    ([1100], [1100], 2, False),                     # pairs
    ([130, 1, 300], [130, 7, 310], 2, True),        # packed, single CTAs
    ([2300, 1900], [2300, 1900], 1, True),          # packed, pairs
    ([300], [4200], 100, False),                    # split over the keys, single CTAs: whole items and parts
    ([1100], [4300], 32, False),                    # split, pairs
    ([1, 130, 300], [5000, 4300, 9000], 2, True),   # packed and split
    ([2100], [9000], 1, True),                      # packed and split, pairs
])
@pytest.mark.parametrize("at", [8, 24])
def test_prefill_writes_an_out_of_any_16_bytes(lq, lk, heads, packed, at):
    """The same bits as into a buffer of the allocator's, and nothing beside it."""
    gen = torch.Generator().manual_seed(sum(lq) + at)
    if not packed:
        assert (M.latent_prefill_workspace_bytes(1, lq[0], lk[0], heads) > 0) == (lk[0] > 4096)
    q, k, pe, v = (_rand(gen, 1, *x).cuda() for x in ((sum(lq), heads, 192), (sum(lk), heads, 128), (sum(lk), 64),
                                                      (sum(lk), heads, 128)))
    cu = [torch.tensor([0] + list(np.cumsum(x)), device="cuda") for x in (lq, lk)] if packed else [None, None]
    lse, again = (torch.full((1, sum(lq), heads), NAN, device="cuda") for _ in range(2))
    ref = M.latent_prefill(q, k, pe, v, 0.07, lse=lse, cu_seqlens=cu[0], cu_seqlens_k=cu[1])
    n = ref.numel()
    buf = torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[at:at + n].view(ref.shape)
    assert ref.data_ptr() % 32 == 0 and out.data_ptr() % 32 == 16
    assert M.latent_prefill(q, k, pe, v, 0.07, out=out, lse=again, cu_seqlens=cu[0], cu_seqlens_k=cu[1]) is out
    assert torch.equal(out, ref) and torch.equal(again, lse)
    assert (buf[:at] == 5.0).all() and (buf[at + n:] == 5.0).all()
    assert get_status() == 0


# ---- refusals of the binding ----

def test_workspaces_that_the_gpu_cannot_write_are_refused():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    decode = z(2, 1, 4, 576), z(80, 8, 576), z(2, 40, d=torch.int32), z(2, d=torch.int32)
    prefill = z(1, 5, 3, 192), z(1, 5, 3, 128), z(1, 5, 64), z(1, 5, 3, 128)
    cu = torch.tensor([0, 5], device="cuda")
    for ws in (torch.empty(1 << 24, dtype=torch.uint8), z(1, d=torch.uint8).expand(1 << 24), z(1 << 24, d=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            M.latent_decode(*decode, 1.0, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            M.latent_prefill(*prefill, 1.0, cu_seqlens=cu, workspace=ws)
    ws = z(1 << 22, d=torch.float32)
    assert torch.equal(M.latent_decode(*decode, 1.0, workspace=ws), M.latent_decode(*decode, 1.0))


@pytest.mark.parametrize("scale", [1e39, float("inf"), float("nan"), -1e39, 0, 1e-60])
def test_scales_that_are_not_positive_32_bit_numbers_are_refused(scale):
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    with pytest.raises(KdaError, match="kda_latent_decode.*16"):
        M.latent_decode(z(2, 1, 4, 576), z(8, 8, 576), z(2, 4, d=torch.int32), z(2, d=torch.int32), scale)
    with pytest.raises(KdaError, match="kda_latent_prefill.*16"):
        M.latent_prefill(z(1, 5, 3, 192), z(1, 5, 3, 128), z(1, 5, 64), z(1, 5, 3, 128), scale)


# ---- the forms that large calls take ----

def _many_lengths(count, longest, seed):
    """Ragged, with empty requests, single tokens, whole tiles and more than four tiles among them."""
    lens = np.random.default_rng(seed).integers(0, longest + 1, count)
    lens[:8] = [0, 1, 64, 128, longest, 0, 0, 65]
    lens[-2:] = [0, longest]
    return [int(x) for x in np.minimum(lens, longest)]


@pytest.mark.parametrize("requests,R,H", [(400, 1, 5), (300, 1, 16), (300, 1, 32), (220, 2, 16), (200, 1, 64), (200, 3, 20),
                                          (160, 1, 128), (120, 2, 65), (90, 3, 64)])
def test_decode_more_requests_than_shares(requests, R, H):
    """Every column width, one and several blocks of query rows: a CTA works on many pieces in turn, and the
    requests that several CTAs hold are listed by share."""
    assert requests > 152 // -(-R * H // 64)
    _decode(_many_lengths(requests, 700, requests + H), R, H, 16, seed=requests)


@pytest.mark.parametrize("requests,R,H", [(400, 1, 8), (333, 2, 16), (170, 1, 64), (120, 3, 64)])
def test_decode_many_short_requests(requests, R, H):
    """Tables of up to four tiles: requests are not split, and there are more of them than CTAs."""
    _decode(_many_lengths(requests, 256, requests), R, H, 64, seed=H)


@pytest.mark.parametrize("T", [4863, 4864, 4865, 14593, 29185])
@pytest.mark.parametrize("norm", [False, True])
def test_append_many_tokens(T, norm):
    """At and past the limit (8 x 152 x 4 tokens) from which a warp takes two at a time, an odd token at the
    end, and past the tokens (912 x 16) that the grid takes in one round; skipped slots and one outside."""
    gen = torch.Generator().manual_seed(T)
    rows = _rand(gen, T, 576, std=2.0).cuda()
    pages = T // 16 + 3
    cache = torch.full((pages, 16, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(pages * 16, generator=gen)[:T]
    slots[torch.randperm(T, generator=gen)[:T // 50]] = -1
    slots[T - 2] = pages * 16
    w = (torch.rand(512, generator=gen) + 0.5).cuda() if norm else None
    M.latent_append(rows[:, :512], rows[:, 512:], slots.cuda(), cache, w, 1e-5)
    assert get_status() == 20  # the slot outside
    kept = (slots >= 0) & (slots < pages * 16)
    flat, at = cache.view(-1, 576), slots[kept].cuda()
    got, src = flat[at], rows[kept.cuda()]
    assert torch.equal(got[:, 512:], src[:, 512:])
    if norm:  # fp32 arithmetic and one rounding to bf16: 2^-8, with 2^-16 for the fp32 steps
        ref = L.normalised(_f64(src[:, :512]), _f64(w), 1e-5)
        assert (np.abs(_f64(got[:, :512]) - ref) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + 1e-38).all()
    else:
        assert torch.equal(got, src)
    rest = torch.ones(pages * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (flat[rest] == 5.0).all()


# ---- graphs whose inputs change between replays ----

@pytest.mark.parametrize("requests,R,H", [(5, 1, 32), (300, 1, 16), (3, 3, 64)])
def test_decode_graph_with_other_lengths(requests, R, H):
    """Lengths are read on the device: every replay answers the lengths of its time, whole buffers anew."""
    gen = torch.Generator().manual_seed(requests)
    most = _many_lengths(requests, 600, 1) if requests > 8 else [900, 2500, 37, 0, 1300][:requests]
    cache, table = _paged(gen, most, 64, behind=0.0)
    q = _rand(gen, requests, R, H, 576)
    dq, dc, dt, lens = q.cuda(), cache.cuda(), table.cuda(), torch.tensor(most, dtype=torch.int32).cuda()
    out = torch.empty(requests, R, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(requests, R, H, device="cuda")
    ws = torch.empty(max(1, M.latent_decode_workspace_bytes(requests, R, H, dc, dt)), dtype=torch.uint8, device="cuda")
    M.latent_decode(dq, dc, dt, lens, 0.07, out, lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.latent_decode(dq, dc, dt, lens, 0.07, out, lse, workspace=ws)
    for now in (most, [n // 2 for n in most], [0] * requests, [min(n, 1) for n in most],
                [n if i % 3 else 0 for i, n in enumerate(most)], most):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(NAN)
        lse.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, L.absorbed(_f64(q), _f64(cache), table.tolist(), now, 0.07), max(now + [1]))
    assert get_status() == 0


@pytest.mark.parametrize("n,keys,heads,offsets", [
    (300, 13000, 2, [([0, 20, 290, 300], [0, 5000, 12000, 13000]), ([0, 0, 1, 300], [0, 12990, 12990, 13000]),
                     ([0, 300, 300, 300], [0, 13000, 13000, 13000])]),           # split over the keys
    (500, 700, 3, [([0, 1, 130, 500], [0, 200, 330, 700]), ([0, 500, 500, 500], [0, 700, 700, 700]),
                   ([0, 200, 400, 500], [0, 10, 600, 700])]),                    # not split
])
def test_packed_prefill_graph_with_other_offsets(n, keys, heads, offsets):
    gen = torch.Generator().manual_seed(n)
    q, k, pe, v = (_rand(gen, 1, *x) for x in ((n, heads, 192), (keys, heads, 128), (keys, 64), (keys, heads, 128)))
    dev = [t.cuda() for t in (q, k, pe, v)]
    cu, cu_k = (torch.tensor(x, device="cuda") for x in offsets[0])
    out, lse = torch.empty(1, n, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, heads, device="cuda")
    ws = torch.empty(M.latent_prefill_workspace_bytes(1, n, keys, heads, 3), dtype=torch.uint8, device="cuda")
    M.latent_prefill(*dev, 0.07, out, lse, cu, cu_k, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.latent_prefill(*dev, 0.07, out, lse, cu, cu_k, workspace=ws)
    for a, b in offsets:
        cu.copy_(torch.tensor(a))
        cu_k.copy_(torch.tensor(b))
        out.fill_(NAN)
        lse.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, L.expanded(_f64(q), _f64(k), _f64(pe), _f64(v), 0.07, True, a, b), keys)
    assert get_status() == 0


@pytest.mark.parametrize("n,keys,heads", [(200, 5000, 2), (1100, 6000, 1), (1100, 1100, 1)])
def test_dense_prefill_graph_with_other_inputs(n, keys, heads):
    """Split in single CTAs, split in pairs, and not split."""
    gen = torch.Generator().manual_seed(keys)
    shapes = (n, heads, 192), (keys, heads, 128), (keys, 64), (keys, heads, 128)
    dev = [torch.zeros(1, *x, dtype=torch.bfloat16, device="cuda") for x in shapes]
    out, lse = torch.empty(1, n, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, heads, device="cuda")
    need = M.latent_prefill_workspace_bytes(1, n, keys, heads)
    assert (need > 0) == (keys > 4096)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    M.latent_prefill(*dev, 0.07, out, lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.latent_prefill(*dev, 0.07, out, lse, workspace=ws)
    for _ in range(2):
        now = [_rand(gen, 1, *x) for x in shapes]
        for d, x in zip(dev, now):
            d.copy_(x)
        out.fill_(NAN)
        lse.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, L.expanded(*(_f64(x) for x in now), 0.07, True), keys)
    assert get_status() == 0
