"""Lists of pages that break the rules, of any length: what counts is attended to wherever it stands in the list, and
everything that does not is flagged."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa_gb300 as csa
from kv8_ref import Cache, Device, bf16

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


def counts(entries, last):
    """(pages that count, whether one that does not stands among them): ascending, up to the row's page, until -1."""
    got, bad = [], False
    for e in entries:
        if e < 0:
            break
        if e > last or (got and e <= got[-1]):
            bad = True
        else:
            got.append(int(e))
    return got, bad


def attend_and_check(s, pos, lists, heads, per=None):
    c = s.c
    lists = np.asarray(lists, np.int32)
    q = bf16(c.rng.standard_normal((len(pos), heads, c.d)))
    out, lse = s.attend([0] * len(pos), pos, q, lists, per=per)
    found = [[counts(lists[r, h], p // 64) for h in range(c.H)] for r, p in enumerate(pos)]
    assert s.flags[1] == (csa.FLAG_TOPK_OOB if any(bad for row in found for _, bad in row) else 0)
    s.check([0] * len(pos), pos, q, out, lse, [[got for got, _ in row] for row in found])


def test_what_counts():
    assert counts([0, 0, 1, -1], 1) == ([0, 1], True)
    assert counts([3, 9, 4, 2, -1, 7], 5) == ([3, 4], True)
    assert counts([0, 1, -1], 5) == ([0, 1], False)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [4, 16, 40])
def test_entries_that_do_not_count_keep_none_out(d, G):
    """Rows of fewer pages than their lists have entries."""
    c = Cache(d + G, [200], 1, d)
    s = Device(csa, c)
    for pos, entries in ((100, [0, 0, 1, -1]), (100, [5, 6, 7, 0, 1, -1]), (10, [1, 2, 3, 4, 5, 0]), (150, [2, 1, 0, 2, 1]),
                         (150, [0] * 40 + [1] * 40 + [2] * 40), (150, [9] * 255 + [0]), (150, [9] * 254 + [0, 2]),
                         (64, [7] * 32 + [0] + [7] * 31 + [1] + [7] * 31 + [-1, 2])):
        attend_and_check(s, [pos], [[entries]], G)


@gpu
@pytest.mark.parametrize("G", [4, 40])
def test_every_entry_is_looked_at(G):
    """A bad entry behind all that a row can hold, in any chunk of the list; none behind -1."""
    c = Cache(7 + G, [64 * 66], 1, 64)
    s = Device(csa, c)
    for pages, more in ((32, [40]), (32, [0]), (64, [64]), (64, [-1, 64, 0]), (1, [0]), (66, [3]), (31, [31])):
        attend_and_check(s, [64 * pages - 1], [[list(range(pages)) + more]], G)
    attend_and_check(s, [100], [[[0, 1] + [-1] * 60 + [5, 5]]], G)
    attend_and_check(s, [100], [[[0, 1] + [1] * 130]], G)


@gpu
@pytest.mark.parametrize("G", [1, 8, 33])
@pytest.mark.parametrize("n,M", [(300, 64), (5000, 100), (20000, 256)])
def test_any_entries(G, n, M):
    """Random lists, falling and repeated entries and pages past the row's own among them, several rows and heads."""
    c = Cache(G + M, [n], 2, 64)
    s = Device(csa, c)
    rng = np.random.default_rng(n + G)
    pos = sorted(int(x) for x in rng.integers(0, n, 5)) + [n - 1]
    lists = np.full((len(pos), 2, M), -1, np.int32)
    for r, p in enumerate(pos):
        for h in range(2):
            k = rng.integers(1, M + 1)
            row = np.sort(rng.integers(0, p // 64 + 2, k)) if (r + h) % 2 else np.sort(rng.choice(n, min(k, n), replace=False) % (p // 64 + 1))
            swap = rng.random(len(row)) < 0.15
            row[swap] = rng.integers(0, n // 32 + 9, swap.sum())
            lists[r, h, :len(row)] = row
    attend_and_check(s, pos, lists, 2 * G)
    attend_and_check(s, pos[-1:], lists[-1:], 2 * G)
