"""csa_dense_attn where several rows of a request share their keys: a group's
window fills two tiles there, and a share of the work may begin at the second."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa_gb300 as csa
from dense_ref import Case, e4m3

gpu = pytest.mark.gpu
WIN, TILE = 128, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


def rope_tables(rows, seed=5):
    th = np.random.default_rng(seed).uniform(0, 2 * np.pi, (rows, 32))
    return np.cos(th).astype(np.float32), np.sin(th).astype(np.float32)


def shares_at_second_window_tile(ctx, r, H, P, sms):
    """The first rows of the groups of whose tiles a CTA's share begins with the
    second one, a window tile, and goes on to entries (the kernel's list of work:
    a group with a window costs its tiles and 6 units, which the last one saves)."""
    cols = 16
    while cols < 64 and cols < r * H:
        cols *= 2
    G = max(cols, H) // H
    groups = []
    for b, c in enumerate(ctx):
        for k in range(0, r, G):
            p0, g = c - r + k, min(G, r - k)
            W = p0 + g - max(0, p0 - WIN + 1)
            Wp = -(-W // TILE) * TILE
            groups.append((b * r + k, Wp, -(-(Wp + (p0 + g) // P) // TILE)))
    ends = np.cumsum([t + 6 for _, _, t in groups])
    per = -(-(int(ends[-1]) - 6) // sms)
    rows = []
    for lo in range(0, int(ends[-1]), per):
        i = int(np.searchsorted(ends, lo, side="right"))
        r0, Wp, tiles = groups[i]
        if lo - (int(ends[i]) - tiles - 6) == 1 and Wp == 2 * TILE and tiles > 2 and per > 1:
            rows.append(r0)
    return rows


def common_block(c):
    """Dims 0..15 of every key are 1."""
    c.kv[:, (256 * np.arange(64)[:, None] + np.arange(8)).ravel()] = 0x22
    c.kv[:, 16384 + 32 * np.arange(64)] = 0x38
    c.wscale[:] = 2.0 ** -6
    c.codes[..., :16] = 0x68


@gpu
@pytest.mark.parametrize("P", [1, 2])
@pytest.mark.parametrize("H,r,B,rope", [(32, 2, 16, False), (32, 3, 16, False), (32, 128, 4, False), (16, 2, 16, False),
                                        (16, 3, 16, False), (16, 4, 16, True), (16, 6, 16, False)])
def test_logits_far_below_zero_where_a_share_begins_in_the_window(H, r, B, rope, P):
    """Softmax does not see a shift of all logits, whatever tile a row meets first."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for more in range(0, 4096, 64):
        ctx = [2050 * P + more + b for b in range(B)]
        cut = shares_at_second_window_tile(ctx, r, H, P, sms)
        if cut:
            break
    assert cut
    c = Case(300 + H + r + P, ctx, P, WIN + r - 1)
    common_block(c)
    req = [b for b in range(B) for _ in range(r)]
    pos = [p for b in range(B) for p in range(ctx[b] - r, ctx[b])]
    tab = rope_tables(max(ctx)) if rope else None
    scale = 512 ** -0.5
    rows = sorted({row for r0 in cut[:4] for row in range(r0, min(r0 + 4, B * r))} | {0, B * r - 1})
    for shift in (28, 60, 200):                           # log2 units
        q = c.queries(B * r, H, 0.3)
        q[..., :16] = -shift * np.log(2) / (16 * scale)
        assert c.run(csa, req, pos, H, q, scale=scale, rope=tab) == (0, 0)
        c.check(req, pos, H, q, scale=scale, rope=tab, rows=rows)


@gpu
@pytest.mark.parametrize("H,r", [(64, 1), (32, 2), (16, 4)])
def test_rotated_window_tokens_at_the_largest_scales(H, r):
    """Codes of 448 in both halves of a rotated pair under scales up to 2^8."""
    ctx = [300, 131, 40]
    c = Case(400 + H, ctx, 2, 140)
    sign = c.g.integers(0, 2, (3, 140, 64), dtype=np.uint8) * 128
    c.codes[..., 448:] = 0x7E + sign
    c.wscale[:] = np.exp2(c.g.uniform(6, 7.999, c.wscale.shape))
    c.wscale[0] = np.float32(255.99)
    req = [b for b in range(3) for _ in range(r)]
    pos = [p for b in range(3) for p in range(ctx[b] - r, ctx[b])]
    q = c.queries(3 * r, H, 1e-4)
    tab = rope_tables(300)
    assert c.run(csa, req, pos, H, q, rope=tab) == (0, 0)
    c.check(req, pos, H, q, rope=tab)


@gpu
@pytest.mark.parametrize("log2", [13.0, 13.97, 13.9999, 14.1])
def test_weights_at_the_largest_step_of_the_maximum(log2):
    """The second window tile's keys exceed the first's by as much as lets the
    maximum stay, or a little more, under the largest window scale.  Enough
    requests for both tiles to be one share's in most of them."""
    B = 300
    c = Case(420, [400] * B, 2, 140)
    c.kv[:, 16384:] = 0                                   # entries of zeros
    c.wscale[:] = np.float32(255.99)
    c.codes[..., 0] = 0
    c.codes[:, np.arange(397, 400) % 140, 0] = 0x68       # 64
    c.codes[..., 448:] = 0x7E
    q = torch.zeros(4 * B, 16, 512, dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** -6
    scale = log2 * np.log(2) / (255.99 * 64 * 2.0 ** -6)
    tab = rope_tables(400)
    req, pos = [b for b in range(B) for _ in range(4)], [396, 397, 398, 399] * B
    assert c.run(csa, req, pos, 16, q, scale=scale, rope=tab) == (0, 0)
    c.check(req, pos, 16, q, scale=scale, rope=tab, rows=list(range(0, 4 * B, 23)) + [4 * B - 1])


@gpu
@pytest.mark.parametrize("H,r", [(32, 2), (16, 4)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_token_without_a_finite_scale_stays_with_the_rows_that_see_it(H, r, bad):
    """The last of a request's new tokens has overflowed: the rows before it do not see it."""
    ctx = [700, 40, 131]
    c = Case(500 + H, ctx, 2, 140)
    for b, n in enumerate(ctx):
        c.wscale[b, (n - 1) % 140] = bad
    req = [b for b in range(3) for _ in range(r)]
    pos = [p for b in range(3) for p in range(ctx[b] - r, ctx[b])]
    q = c.queries(3 * r, H)
    assert c.run(csa, req, pos, H, q) == (0, 0)
    last = [r - 1, 2 * r - 1, 3 * r - 1]
    c.check(req, pos, H, q, rows=[i for i in range(3 * r) if i not in last])
    assert c.out[last].isnan().all() and c.lse[last].isnan().all()


@gpu
@pytest.mark.parametrize("rope", [False, True])
def test_negative_window_scales(rope):
    """A token is its codes times its scale, whatever the scale's sign."""
    c = Case(510, [500, 90], 2, 140)
    c.wscale *= np.where(c.g.random(c.wscale.shape) < 0.5, np.float32(-1), np.float32(1))
    req, pos = [0, 0, 1, 1], [498, 499, 88, 89]
    q = c.queries(4, 32)
    tab = rope_tables(500) if rope else None
    assert c.run(csa, req, pos, 32, q, rope=tab) == (0, 0)
    c.check(req, pos, 32, q, rope=tab)


@gpu
def test_tiny_window_scales_lose_no_more_than_stated():
    """Tokens alone (no entry yet) under scales of 2^-34: P is subnormal, and off
    by half its step, 2^-25, times codes of 2^-14."""
    c = Case(430, [1], 2, 128)
    c.wscale[:] = np.float32(2.0 ** -34)
    q = c.queries(1, 32)
    assert c.run(csa, [0], [0], 32, q) == (0, 0)
    want = e4m3(c.codes[0, 0]) * 2.0 ** -34
    err = np.abs(c.out[0].double().cpu().numpy() - want)
    assert (err <= 2.0 ** -39 * np.abs(want) * 2.0 ** 34 + 2.0 ** -8 * np.abs(want)).all()


@gpu
def test_query_elements_far_below_the_largest():
    """One element 2^16 times the others, against zeros in every key."""
    c = Case(440, [900, 70], 1, 128)
    c.kv[:, 256 * np.arange(64)] &= 0xF0
    c.codes[..., 0] = 0
    q = c.queries(2, 32)
    q[..., 0] = 2.0 ** 16
    assert c.run(csa, [0, 1], [899, 69], 32, q) == (0, 0)
    c.check([0, 1], [899, 69], 32, q)
