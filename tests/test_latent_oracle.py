"""Pins of oracle/latent.py to facts that do not come from it."""
import math

import numpy as np
import pytest

from oracle import latent as L

RNG = np.random.default_rng(5)


def _paged(rows, lens, page):
    """Rows of every request laid into a shuffled paged cache; returns cache, table."""
    need = [-(-n // page) for n in lens]
    perm = RNG.permutation(sum(need) + 2)
    cache = RNG.standard_normal((sum(need) + 2, page, rows[0].shape[1]))
    table = np.zeros((len(lens), max(need + [1])), np.int64)
    at = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = perm[at]
            part = rows[b][j * page:(j + 1) * page]
            cache[perm[at], :len(part)] = part
            at += 1
    return cache, table


@pytest.mark.parametrize("R", [1, 3])
def test_absorbed_and_expanded_forms_agree(R):
    """k_h = W_uk c, v_h = W_uv c: the absorbed query [W_uk^T q | q_pe] and W_uv applied to the
    absorbed output give the expanded result (the products are associative), and the same lse."""
    H, lens, page = 2, [5, 17], 8
    w_uk, w_uv = RNG.standard_normal((2, H, 128, 512)) / 20
    rows = [RNG.standard_normal((n, 576)) for n in lens]
    q = RNG.standard_normal((len(lens), R, H, 192))
    cache, table = _paged(rows, lens, page)
    q_abs = np.concatenate([np.einsum("brhd,hdc->brhc", q[..., :128], w_uk), q[..., 128:]], -1)
    o, lse, _, _ = L.absorbed(q_abs, cache, table, lens, 0.07)
    o = np.einsum("brhc,hdc->brhd", o, w_uv)
    for b, n in enumerate(lens):
        c, pe = rows[b][:, :512], rows[b][:, 512:]
        k, v = np.einsum("tc,hdc->thd", c, w_uk), np.einsum("tc,hdc->thd", c, w_uv)
        ref, ref_lse, _, _ = L.expanded(q[b:b + 1], k[None], pe[None], v[None], 0.07, True)
        assert np.allclose(o[b], ref[0], rtol=1e-11, atol=1e-11)
        assert np.allclose(lse[b], ref_lse[0], rtol=1e-12, atol=1e-12)


def test_zero_queries_average_the_values():
    """q = 0: uniform weights; out = mean of the visible values, lse = ln(count)."""
    v = RNG.standard_normal((1, 6, 1, 128))
    z = np.zeros((1, 4, 1, 192))
    o, lse, spread, reach = L.expanded(z, RNG.standard_normal((1, 6, 1, 128)), RNG.standard_normal((1, 6, 64)), v, 1.0, True)
    for i in range(4):  # query i sees 6 - 4 + i + 1 keys
        assert np.allclose(o[0, i, 0], v[0, :3 + i, 0].mean(0), atol=1e-14)
        assert math.isclose(lse[0, i, 0], math.log(3 + i), rel_tol=1e-14)
        assert np.allclose(spread[0, i, 0], np.abs(v[0, :3 + i, 0]).mean(0), atol=1e-14)
    assert (reach == 0).all()


def test_rows_that_see_nothing():
    o, lse, _, _ = L.expanded(np.ones((1, 3, 1, 192)), np.ones((1, 1, 1, 128)), np.ones((1, 1, 64)),
                              np.ones((1, 1, 1, 128)), 1.0, True)
    assert (o[0, :2] == 0).all() and np.isneginf(lse[0, :2]).all() and np.allclose(o[0, 2], 1)
    o, lse, _, _ = L.absorbed(np.ones((1, 2, 1, 576)), np.ones((1, 8, 576)), [[0]], [1], 1.0)
    assert (o[0, 0] == 0).all() and np.isneginf(lse[0, 0]).all() and np.allclose(o[0, 1], 1)


def test_chunks_of_keys_join_through_lse():
    """softmax over a union = the parts weighted by exp(lse_part - lse)."""
    q = RNG.standard_normal((1, 2, 1, 192))
    k, pe, v = (RNG.standard_normal(s) for s in ((1, 9, 1, 128), (1, 9, 64), (1, 9, 1, 128)))
    o, lse, _, _ = L.expanded(q, k, pe, v, 0.1, False)
    a, za, _, _ = L.expanded(q, k[:, :4], pe[:, :4], v[:, :4], 0.1, False)
    b, zb, _, _ = L.expanded(q, k[:, 4:], pe[:, 4:], v[:, 4:], 0.1, False)
    assert np.allclose(np.logaddexp(za, zb), lse, rtol=1e-13)
    assert np.allclose(np.exp(za - lse)[..., None] * a + np.exp(zb - lse)[..., None] * b, o, atol=1e-13)


def test_plan_by_hand():
    p = L.plan([0, 8, 5, 0], [9, 1, 2, 0], [[0] * 3 for _ in range(2)] + [[7, 0, 0], [0] * 3],
               [10, 11, 12, 13], 8, 14)
    assert p["table"][0][:2] == [10, 11] and p["table"][1] == [0, 12, 0] and p["table"][2] == [7, 0, 0]
    assert p["seq_lens"] == [9, 9, 7, 0] and p["cu_seqlens"] == [0, 9, 10, 12, 12] and p["pages_taken"] == [3]
    assert p["slot_map"] == list(range(80, 88)) + [88, 96, 61, 62, -1, -1]


def test_normalised_rows_have_unit_mean_square():
    y = L.normalised(RNG.standard_normal((4, 512)) * 30, np.ones(512), 0.0)
    assert np.allclose((y ** 2).mean(1), 1, rtol=1e-12)
