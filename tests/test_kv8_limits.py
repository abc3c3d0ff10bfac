"""The 8-bit cache's calls at the ends of their arguments' ranges."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa_gb300 as csa
from kv8_ref import Cache, Device, bf16

gpu = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


@pytest.mark.parametrize("op", [csa.OP_KV8_ATTN, csa.OP_KV8_SELECT])
@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 32), (6, 64), (64, 64)])
def test_workspace_does_not_shrink_up_to_the_largest_bound(op, rows, heads):
    sizes = [csa.csa_workspace_size(op, rows, n, heads) for n in (1, 1 << 20, 1 << 30, MOST - 63, MOST - 62, MOST)]
    assert sizes == sorted(sizes)
    assert sizes[-1] < 1 << 40


@gpu
@pytest.mark.parametrize("rows,G", [(1, 8), (9, 8)])
def test_rows_bounded_by_all_positions_there_are(rows, G):
    """A page table as wide as positions allow, and max_entries to match: the same results, in a workspace as
    large as for any long row."""
    c = Cache(5 + rows, [3000], 2, 64)
    s = Device(csa, c)
    pos = list(range(3000 - rows, 3000))
    q = bf16(c.rng.standard_normal((rows, 2 * G, 64)))
    wide = torch.full((1, 1 << 25), -1, dtype=torch.int32, device="cuda")
    wide[0, :s.table.shape[1]] = s.table[0]
    s.cache = csa.make_kv8(s.pool, s.tail, wide, c.pages, 2, 64)
    out, lse = s.attend([0] * rows, pos, q, most=MOST)
    assert s.flags == (0, 0)
    s.check([0] * rows, pos, q, out, lse, rows=[0, rows - 1])
    long, lse2 = s.attend([0] * rows, pos, q, most=1 << 20)
    assert np.array_equal(out, long) and np.array_equal(lse, lse2)


@gpu
@pytest.mark.parametrize("rows,G", [(1, 4), (2, 8), (4, 7), (3, 16), (20, 8), (9, 33)])
@pytest.mark.parametrize("qs,ks,scale", [(300.0, 300.0, 1.0), (1e4, 1e4, 0.1), (1e6, 1e6, 1.0), (1e15, 1e15, 1.0), (1.0, 1.0, 1e25),
                                         (1e4, 1e4, -0.1)])
def test_logits_of_any_size(rows, G, qs, ks, scale):
    """The largest logit 2^18 to 2^120, the next one far below it, or equal to it to the last bit: the output is the value
    of the first, or the mean of the two, and the sum's logarithm that logit."""
    d, n = 64, 700
    rng = np.random.default_rng(rows + G)
    k = np.sign(rng.standard_normal((n, 1, d))) * ks
    v = bf16(rng.standard_normal((n, 1, d)))
    for twins in (False, True):
        q = np.empty((rows, G, d), np.float32)
        best = rng.integers(0, n - rows, (rows, G))
        other = (best + 64 * rng.integers(1, 9, (rows, G))) % (n - rows)
        kk = k.copy()
        if twins:
            best[:], other[:] = 37, 437
            kk[437] = kk[37]
        kk = bf16(kk)
        for r in range(rows):
            for g in range(G):
                q[r, g] = np.sign(kk[best[r, g], 0]) * (qs if scale > 0 else -qs)
        q = bf16(q)
        c = Cache(1, [n], 1, d, tokens=[(kk, v)])
        s = Device(csa, c)
        pos = list(range(n - rows, n))
        out, lse = s.attend([0] * rows, pos, q, scale=scale)
        assert s.flags == (0, 0)
        pool = s.pool.cpu().numpy()
        from kv8_ref import head_entries
        key, val, _ = head_entries(pool, c.table[0], 0, d, np.arange(-(-n // 64)))
        for r in range(rows):
            x = (q[r].astype(np.float64) @ key[:pos[r] + 1].T) * scale
            top = x.max(-1)
            gap = top - np.where(np.arange(pos[r] + 1)[None] == best[r][:, None], -np.inf,
                                 np.where(twins & (np.arange(pos[r] + 1) == 437), -np.inf, x)).max(-1)
            assert (np.argmax(x, -1) == best[r]).all() and (gap > 2.0 ** -3 * np.abs(top)).all()   # keys' signs agree in some dims only
            assert np.isfinite(lse[r]).all() and (np.abs(lse[r] - top) <= 1 + 2.0 ** -17 * np.abs(top)).all(), (r, lse[r], top)
            want = (val[37] + val[437]) / 2 if twins else val[best[r]]
            if twins and np.abs(top).max() < 2.0 ** 20:      # both in one fp32 difference
                assert (np.abs(out[r] - want) <= 2.0 ** -6 * (1 + np.abs(want))).all()
            elif twins:                                      # any mean of the two
                lo, hi = np.minimum(val[37], val[437]), np.maximum(val[37], val[437])
                assert ((out[r] >= lo - 2.0 ** -6 * (1 + np.abs(lo))) & (out[r] <= hi + 2.0 ** -6 * (1 + np.abs(hi)))).all()
            else:
                assert (np.abs(out[r] - want) <= 2.0 ** -7 * (1 + np.abs(want))).all()


@gpu
@pytest.mark.parametrize("seed", range(4))
def test_drafts_rejected_time_and_again(seed):
    """Appends from anywhere down to 64 below the highest position that was ever written: in the end pages, summaries
    and tail are those of the tokens that stayed."""
    n = 700
    c = Cache(30 + seed, [n], 2, 64)
    s = Device(csa, c, filled=False)
    rng = np.random.default_rng(seed)
    kept = most = calls = 0                                # tokens that stay; one past the highest position written
    while kept < n:
        lo = int(rng.integers(max(0, most - 64), kept + 1)) if calls % 2 else kept
        new = int(min(rng.integers(1, 65), n - lo))
        stay = new if calls % 3 == 0 else int(rng.integers(0, new + 1))
        s.append([lo], [new], *(np.concatenate([x[lo:lo + stay], bf16(rng.standard_normal((new - stay, 2, 64)))])
                                for x in c.tokens[0]))
        kept, most, calls = lo + stay, max(most, lo + new), calls + 1
    assert s.status() == (0, 0) and calls > 20
    pool, codes, scale, tail = c.fill()
    assert np.array_equal(s.pool.cpu().numpy(), pool)
    assert np.array_equal(s.codes.cpu().numpy(), codes) and np.array_equal(s.scale.cpu().numpy(), scale)
    assert np.array_equal(s.tail.float().cpu().numpy(), tail)


@gpu
@pytest.mark.parametrize("rows,G", [(1, 4), (4, 7), (3, 16), (20, 8), (9, 33)])
@pytest.mark.parametrize("scale", [1.0, 1e6, 1e12])
@pytest.mark.parametrize("at", [3, 400, 690])
def test_no_number_among_logits_of_any_size(rows, G, scale, at):
    """Rows that see a token with a NaN or an infinity become NaN, and no others, beside small logits and large ones,
    alike scales and far ones."""
    d, n = 64, 700
    rng = np.random.default_rng(at)
    for far in (False, True):
        k, v = bf16(rng.standard_normal((n, 1, d)) * 30), bf16(rng.standard_normal((n, 1, d)))
        if far:
            v = bf16(v * 10.0 ** rng.integers(-9, 9, -(-n // 64))[np.arange(n) // 64][:, None, None])
        k[at, 0, 7], v[at + 1, 0, 3] = np.nan, np.inf
        s = Device(csa, Cache(2, [n], 1, d, tokens=[(k, v)]))
        pos = [int(x) for x in np.concatenate([np.arange(n - rows, n), np.arange(at - 2, at + 3)]) if x >= 0]
        q = bf16(rng.standard_normal((len(pos), G, d)) * 30)
        out, lse = s.attend([0] * len(pos), pos, q, scale=scale)
        assert s.flags == (0, 0)
        sees = np.array(pos) >= at
        assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all()
        assert np.isfinite(out[~sees]).all() and np.isfinite(lse[~sees]).all()


@gpu
@pytest.mark.parametrize("rows,G", [(1, 4), (1, 16), (1, 32), (4, 7), (20, 8), (9, 33)])
@pytest.mark.parametrize("scale", [1.0, 1e3, 1e6, 1e20])
@pytest.mark.parametrize("n", [120, 700])
def test_large_logits_beside_far_scales(rows, G, scale, n):
    """The value of the one key above all others, to the last bits, whatever its page's scale and the others' are."""
    d = 64
    rng = np.random.default_rng(rows + G + n)
    k = bf16(np.sign(rng.standard_normal((n, 1, d))) * 30.0)
    for span in (0, 5, 25):
        v = bf16(rng.standard_normal((n, 1, d)) * 10.0 ** rng.uniform(-span, span, -(-n // 64))[np.arange(n) // 64][:, None, None])
        if span == 5:
            v[64:128] = 0
        best = rng.integers(0, n - rows, (rows, G))
        q = bf16(np.sign(k[best, 0]) * 30.0)
        s = Device(csa, Cache(1, [n], 1, d, tokens=[(k, v)]))
        pos = list(range(n - rows, n))
        out, lse = s.attend([0] * rows, pos, q, scale=scale)
        assert s.flags == (0, 0)
        from kv8_ref import head_entries
        key, val, _ = head_entries(s.pool.cpu().numpy(), s.c.table[0], 0, d, np.arange(-(-n // 64)))
        for r in range(rows):
            x = (q[r].astype(np.float64) @ key[:pos[r] + 1].T) * scale
            assert (x.argmax(-1) == best[r]).all()
            # the others' weights are 2^-5000 and less
            want = val[best[r]]
            assert (np.abs(out[r] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max(-1, keepdims=True)).all(), (span, r)
            assert (np.abs(lse[r] - x.max(-1)) <= 2.0 ** -17 * x.max(-1)).all()
