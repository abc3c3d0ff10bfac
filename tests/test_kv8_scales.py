"""Attention over pages of the 8-bit cache whose value scales lie far apart, or that hold no values at all: outputs and
sums against 64 bits, in groups of few and of many columns, whole rows and rows that are cut over the GPU."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa_gb300 as csa
from kv8_ref import PAGE, RING, Cache, Device, bf16, dev, head_entries

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


def attend(pool, table_row, h, d, pos, q, scale, pages=None):
    """(out [G, d], lse [G], bounds of both) of one row and key head in float64, q [G, d].

    The bounds are those of the roundings that the calls state.  A query above 2^-9 of its largest element is exact,
    below that 2^-17 of the largest is lost; a product's fp32 sums 2^-18 of the sum of magnitudes; a logit's factors
    and its difference to a maximum 2^-21 of it and 2^-23 of the column's largest; powers of two, their sum and its
    logarithm 2^-20 + n 2^-31.  A probability times its value's scale is kept to 2^-11 of itself and 2^-24 of the
    row's largest such product, to which a page of no values adds nothing.  The output's sums 2^-18, its rounding to bf16
    2^-8 and, of what bf16 no longer holds, half of its smallest step."""
    pages = np.arange(pos // PAGE + 1) if pages is None else np.asarray(pages)
    see = (pages[:, None] * PAGE + np.arange(PAGE)).reshape(-1) <= pos
    k, v, sc = head_entries(pool, table_row, h, d, pages)
    k, v, sv = k[see], v[see], np.repeat(sc[:, 1], PAGE)[see]
    q = np.asarray(q, np.float64)
    x = (q @ k.T) * scale
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    L = p.sum(-1, keepdims=True)
    lse, w = (m + np.log(L))[:, 0], p / L
    out = w @ v
    top = np.abs(q).max(-1, keepdims=True)
    lost = 2.0 ** -17 * top * (np.abs(q) < 2.0 ** -9 * top)
    dx = abs(scale) * (lost @ np.abs(k).T + 2.0 ** -18 * (np.abs(q) @ np.abs(k).T)) + 2.0 ** -21 * np.abs(x)
    dx = dx.max(-1) + 2.0 ** -23 * np.abs(m[:, 0])
    dl = dx + 2.0 ** -20 + len(k) * 2.0 ** -31 + 2.0 ** -22 * np.abs(lse)
    code = np.abs(v) / np.where(sv > 0, sv, 1.0)[:, None]                 # zeros in a page of no values
    do = (2.0 ** -11 + 2.0 ** -18 + 2 * dl[:, None]) * (w @ np.abs(v)) + 2.0 ** -24 * (w * sv).max(-1, keepdims=True) * code.sum(0)
    return out, lse, do + 2.0 ** -8 * (np.abs(out) + do) + 2.0 ** -134, dl


def check(s, req, pos, q, out, lse, rows=None, lists=None):
    d, H = s.c.d, s.c.H
    G = q.shape[1] // H
    pool, table = s.pool.cpu().numpy(), s.table.cpu().numpy()
    assert s.flags == (0, 0)
    for r in range(len(req)) if rows is None else rows:
        for h in range(H):
            at = slice(h * G, h * G + G)
            pages = None if lists is None else [j for j in lists[r][h] if j >= 0]
            o, z, do, dz = attend(pool, table[req[r]], h, d, pos[r], bf16(q[r, at]), d ** -0.5, pages)
            assert np.isfinite(out[r, at]).all() and np.isfinite(lse[r, at]).all(), (r, h, pos[r])
            worst = np.abs(out[r, at] - o) / do
            assert (worst <= 1).all(), (r, h, pos[r], float(worst.max()), float(np.abs(o).max()))
            assert (np.abs(lse[r, at] - z) <= dz).all(), (r, h, lse[r, at] - z, dz)


def keys_and_values(seed, n, kv, d, scales, climbs=None):
    """n tokens; page j's values about scales[j] (0: none), its keys' first element climbs[j]."""
    rng = np.random.default_rng(seed)
    pages = -(-n // PAGE)
    at = np.arange(n) // PAGE
    k = rng.standard_normal((n, kv, d)) * 0.05
    k[..., 0] = 0 if climbs is None else np.resize(climbs, pages)[at][:, None]
    v = (rng.standard_normal((n, kv, d)) * 0.25 + 1) * np.resize(scales, pages)[at][:, None, None]
    return bf16(k), bf16(v)


def queries(rng, rows, kv, G, d):
    """Columns that go along with the keys' first element, against it, or hardly look at it."""
    q = bf16(rng.standard_normal((rows, kv * G, d)) * 0.5)
    q[..., 0] = np.resize([8.0, -8.0, 0.25, 8.0, 2.0], kv * G)
    return q


def bits(c, d):
    """The first element of a key that puts a logit c powers of two above one of 0, for a query with 8 there."""
    return c * np.log(2) * np.sqrt(d) / 8


# rows and query heads a key head: 8, 16 and 32 columns; a tile of 128 columns shared by the halves; two tiles
GROUPS = [(1, 4), (2, 8), (4, 7), (3, 16), (20, 8), (9, 33)]


def run(seed, n, rows, G, d, scales, climbs, kv=1, lists=None):
    c = Cache(seed, [n], kv, d, tokens=[keys_and_values(seed, n, kv, d, scales, climbs)])
    s = Device(csa, c)
    pos = list(range(n - rows, n))
    q = queries(c.rng, rows, kv, G, d)
    out, lse = s.attend([0] * rows, pos, q, lists)
    check(s, [0] * rows, pos, q, out, lse, sorted({0, rows // 2, rows - 1}), lists)
    return s, q, out, lse


def long_row(n, kv, d, scales, climbs, rows, G):
    """One request's last rows, its cache filled on the GPU."""
    k, v = keys_and_values(n, n, kv, d, scales, climbs)
    c = Cache(n + G, [n], kv, d, tokens=[(np.zeros((0, kv, d), np.float32),) * 2])
    s = Device.__new__(Device)
    s.csa, s.c, s.rope = csa, c, None
    s.pool = torch.zeros(c.pages, kv, 128 * d + 128, dtype=torch.uint8, device="cuda")
    s.table, s.tail = dev(c.table), torch.zeros(1, kv, 2, RING, d, dtype=torch.bfloat16, device="cuda")
    s.cache = csa.make_kv8(s.pool, s.tail, s.table, c.pages, kv, d)
    csa.csa_kv8_append(s.cache, None, dev(np.zeros(1, np.int32)), dev(np.array([0, n], np.int32)), n, dev(k, torch.bfloat16),
                       dev(v, torch.bfloat16))
    torch.cuda.synchronize()
    pos = list(range(n - rows, n))
    q = queries(c.rng, rows, kv, G, d)
    out, lse = s.attend([0] * rows, pos, q)
    check(s, [0] * rows, pos, q, out, lse, sorted({0, rows - 1}))
    return s, q, out, lse


# ---- values near the end of the range -----------------------------------------------------------
@gpu
@pytest.mark.parametrize("rows,G", [(1, 8), (1, 16), (1, 32), (20, 8)])
@pytest.mark.parametrize("scale", [1e33, 6e37])
def test_large_values_in_cut_rows(rows, G, scale):
    """What parts add up to passes fp32's range unless their weights are small numbers."""
    long_row(12000, 1, 128, [scale], [0.0], rows, G)


# ---- scales far apart -----------------------------------------------------------------------
FAR = [[1e10, 1e-29], [1e30, 1e-15], [1e-25, 1e15], [1e-29, 1e37], [1e30, 1, 1e-20], [1e-20, 1, 1e30],
       [1, 1, 1, 1e-18, 1, 1e18], [1e-9, 1e-9, 1e9, 1e-9]]


@gpu
@pytest.mark.parametrize("rows,G", GROUPS)
@pytest.mark.parametrize("scales", FAR)
def test_value_scales_far_apart(rows, G, scales):
    """Flat logits, and pages of small values that some columns put far above the others, by up to 2^220."""
    for d, n, climbs in ((128, 500, [0.0]), (64, 500, [0.0, bits(220, 64), bits(-60, 64)]), (64, 900, [bits(c, 64) for c in (3, -90, 110)])):
        run(len(scales) + rows + n, n, rows, G, d, scales, climbs)


@gpu
@pytest.mark.parametrize("d,kv,rows,G", [(128, 1, 1, 8), (64, 2, 1, 16), (128, 1, 6, 16)])
def test_value_scales_far_apart_in_cut_rows(d, kv, rows, G):
    """A row's parts, in units of their own, joined; some parts' scales alike, some far apart."""
    n = 12000
    rng = np.random.default_rng(n + rows)
    few = rng.choice([1e30, 1e-20, 1.0, 1e12], -(-n // PAGE), p=[0.02, 0.04, 0.9, 0.04])
    far = 10.0 ** rng.integers(-28, 36, -(-n // PAGE))
    for scales, climbs in ((few, [0.0]), (few, bits(rng.uniform(-70, 70, 188), d)), (far, bits(rng.uniform(-100, 100, 188), d))):
        s, q, out, lse = long_row(n, kv, d, scales, climbs, rows, G)
        again, lse2 = s.attend([0] * rows, list(range(n - rows, n)), q)
        assert np.array_equal(out, again) and np.array_equal(lse, lse2)


# ---- pages of no values -----------------------------------------------------------------------
NONE = [[0, 1e-3], [0, 1e-4, 1e-4], [0, 0, 1e-5], [0, 0, 0, 1e-20], [1, 0, 1, 1], [1e-3, 1e-3, 0, 0], [1.0, 0, 1e-20], [0, 1e30]]


@gpu
@pytest.mark.parametrize("rows,G", GROUPS)
@pytest.mark.parametrize("scales", NONE)
def test_pages_of_no_values(rows, G, scales):
    """First in a row, in its first tile, in the middle and last; their keys as probable as others, or up to 2^150 more or
    less so."""
    for d, n, c in ((128, 500, 0), (64, 500, 7), (64, 700, 15), (128, 380, 150)):
        run(len(scales) + rows + n, n, rows, G, d, scales, [bits(c, d) if x == 0 else 0.0 for x in scales])


@gpu
@pytest.mark.parametrize("rows,G", GROUPS)
def test_rows_that_see_no_values_at_all(rows, G):
    s, q, out, lse = run(rows + G, 300, rows, G, 64, [0.0], [0.0, 1.0])
    assert not out.any()


@gpu
@pytest.mark.parametrize("d,kv,rows,G", [(128, 1, 1, 8), (64, 2, 1, 16), (128, 1, 6, 16)])
def test_pages_of_no_values_in_cut_rows(d, kv, rows, G):
    """Parts that begin with such pages, and some that have no others."""
    n = 12000
    rng = np.random.default_rng(n + rows)
    scales = np.where(rng.random(188) < 0.4, 0.0, 1e-5)
    scales[60:100] = 0
    for climbs in (0 * scales, np.where(scales == 0, bits(9, d), 0.0), bits(rng.uniform(-20, 20, 188), d)):
        long_row(n, kv, d, scales, climbs, rows, G)


@gpu
@pytest.mark.parametrize("rows,G", [(1, 4), (1, 16)])
def test_listed_pages_of_no_values_and_far_scales(rows, G):
    scales = [0, 1e-5, 1e10, 0, 1e-25, 1, 1]
    run(3, 1200, rows, G, 64, scales, [bits(c, 64) for c in (5, 0, -60, 100, 80)], lists=[[[0, 3, 7, 8, 10, 11, 14]]])
    run(4, 1200, rows, G, 64, scales, [0.0], lists=[[[1, 2, 4, 18]]])


@gpu
@pytest.mark.parametrize("rows,G", [(1, 8), (1, 16), (1, 32), (20, 8)])
@pytest.mark.parametrize("scale", [1e-25, 1e-29])
def test_small_values_in_cut_rows(rows, G, scale):
    long_row(12000, 1, 128, [scale], [0.0], rows, G)


@gpu
@pytest.mark.parametrize("rows,G", [(1, 4), (1, 16), (1, 32), (9, 7)])
def test_parts_of_small_weight_and_large_values(rows, G):
    """Parts whose sums are up to 2^-220 of another's and whose values make up for it."""
    for seed in range(24):
        rng = np.random.default_rng(seed)
        n = int(rng.integers(130, 1000))
        pages = -(-n // PAGE)
        run(seed, n, min(rows, n), G, 64, 10.0 ** rng.uniform(-28, 34, pages), bits(rng.uniform(-150, 150, pages), 64))


@gpu
@pytest.mark.parametrize("rows,G", [(1, 8), (6, 16), (40, 8)])
@pytest.mark.parametrize("budget", [200, 3000, 20000])
def test_waits_that_run_out_among_far_scales(rows, G, budget):
    """A short limit for each wait: the call returns whatever it got to, and the next one is right."""
    scales = [1, 1, 0, 1e12, 1, 1e-9, 1, 1]
    s, q, out, lse = long_row(5000, 2, 128, scales, bits(np.array([0, 3, 9, -40, 0, 25]), 128), rows, G)
    pos = list(range(5000 - rows, 5000))
    csa.csa_set_wait_budget(budget)                        # SM clocks; the shortest is less than any copy takes
    try:
        s.attend([0] * rows, pos, q)
        assert s.flags in ((0, 0), (6, csa.FLAG_TIMEOUT)) and (budget > 200 or s.flags[0] == 6)
    finally:
        csa.csa_set_wait_budget(0)
    again, lse2 = s.attend([0] * rows, pos, q)
    assert s.flags == (0, 0) and np.array_equal(out, again) and np.array_equal(lse, lse2)


@gpu
@pytest.mark.parametrize("rows,G", [(160, 8), (96, 16), (70, 33), (40, 5)])
def test_far_scales_in_segments_of_many_tiles(rows, G):
    """More work than there are CTAs: each has whole segments, tile after tile of them far from the first."""
    n, scales = 1400, [1, 1e-3, 0, 1e12, 1, 1e-9, 1, 0, 1e20, 1e-20]
    for climbs in ([0.0], bits(np.array([0, 3, 9, -40, 0, 25, -80]), 64)):
        run(rows + G, n, rows, G, 64, scales, climbs, kv=3)
