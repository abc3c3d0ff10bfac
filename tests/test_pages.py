"""csa_pages_reserve / fork / free / compact against a plain model of a page
table with counts, byte for byte; refusals; a captured step that reserves,
appends and attends; and a run of all of them as a serving loop would use them."""
import ctypes as C

import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa_gb300 as csa

gpu = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


# ---- refusals (no kernel runs) --------------------------------------------------------
def test_refusals_before_any_launch():
    lib = csa.lib()
    buf = (C.c_uint8 * 65536)()
    base = (C.addressof(buf) + 255) & ~255
    pt, other, ints = (C.c_int32 * 4)(), (C.c_int32 * 4)(), (C.c_int32 * 8)()
    cache = csa.CsaCache(base, base, C.addressof(pt), 1, 1, 1, 2)
    good = csa.CsaPages(C.addressof(pt), base)
    i = C.addressof(ints)
    big = 1 << 40

    def calls(c, p, n=1, lst=i, extra=i, ws=base, size=big):
        pc, pp = (C.byref(c) if c else None), (C.byref(p) if p else None)
        return (lib.csa_pages_reserve(pc, pp, n, lst, extra, extra, 4, ws, size, None),
                lib.csa_pages_fork(pc, pp, None, None, n, extra, lst, extra, ws, size, None),
                lib.csa_pages_free(pc, pp, n, lst, None, ws, size, None))

    assert calls(None, good) == (1, 1, 1) and calls(cache, None) == (1, 1, 1)
    for p in (csa.CsaPages(C.addressof(other), base), csa.CsaPages(C.addressof(pt), None),
              csa.CsaPages(C.addressof(pt), base + 4)):
        assert calls(cache, p) == (1, 1, 1)
        assert lib.csa_pages_compact(C.byref(cache), C.byref(p), None, None, base, big, None) == 1
    assert calls(cache, good, n=-1) == (1, 1, 1) and calls(cache, good, lst=None) == (1, 1, 1)
    assert calls(cache, good, extra=None)[:2] == (1, 1)
    assert calls(cache, good, n=0) == (0, 0, 0)
    assert calls(cache, good, size=16) == (3, 3, 3) and calls(cache, good, ws=base + 64) == (3, 3, 3)
    assert lib.csa_pages_reserve(C.byref(cache), C.byref(good), 1, i, i, i, -1, base, big, None) == 1
    assert lib.csa_pages_reserve(C.byref(cache), C.byref(good), 1, i, i, i, 4, None, 0, None) == 3
    assert lib.csa_pages_reserve(C.byref(cache), C.byref(good), 2 ** 20, i, i, i, 2 ** 20, base, big, None) == 2
    assert lib.csa_pages_compact(C.byref(cache), C.byref(good), None, None, None, 0, None) == 3
    assert lib.csa_pages_compact(C.byref(cache), C.byref(good), i + 2, None, base, big, None) == 1
    win = csa.CsaWindow(base, base, 100)
    assert lib.csa_pages_fork(C.byref(cache), C.byref(good), C.byref(win), None, 1, i, i, i, base, big, None) == 1
    assert lib.csa_pages_fork(C.byref(cache), C.byref(good), None, base + 8, 1, i, i, i, base, big, None) == 1


def test_short_lists_are_refused():
    cache, pages = csa.CsaCache(), csa.CsaPages()
    three, two = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(csa.CsaError):
        csa.csa_pages_reserve(cache, pages, three, two, three, 4, None, 0)
    with pytest.raises(csa.CsaError):
        csa.csa_pages_fork(cache, pages, None, None, two, three, three, None, 0)
    with pytest.raises(csa.CsaError):
        csa.csa_pages_free(cache, pages, three, two, None, 0)


# ---- the model ------------------------------------------------------------------------
class Model:
    def __init__(self, table, refs, kv, idx):
        self.table, self.refs, self.kv, self.idx = table.copy(), refs.copy(), kv.copy(), idx.copy()

    def reserve(self, req, first, count):
        refs0 = self.refs.copy()
        free = [int(p) for p in np.nonzero(refs0 <= 0)[0]]
        short = False
        for b, f, n in zip(req, first, count):
            if b < 0 or n == 0:
                continue
            for lp in range(f // PAGE, (f + n - 1) // PAGE + 1):
                old = self.table[b, lp]
                if old >= 0 and refs0[old] == 1:
                    continue
                if not free:
                    short = True
                    continue
                new = free.pop(0)
                if old >= 0:
                    self.kv[new], self.idx[new] = self.kv[old], self.idx[old]
                    self.refs[old] -= 1
                self.refs[new] = 1
                self.table[b, lp] = new
        return csa.FLAG_NO_PAGES if short else 0

    def fork(self, parent, child, entries):
        for p, c, n in zip(parent, child, entries):
            if c < 0:
                continue
            for old in self.table[c]:
                if old >= 0:
                    self.refs[old] -= 1
            k = -(-n // PAGE)
            self.table[c] = -1
            self.table[c, :k] = self.table[p, :k]
            for new in self.table[c]:
                if new >= 0:
                    self.refs[new] += 1

    def free(self, req, keep):
        for b, n in zip(req, keep):
            if b < 0:
                continue
            for j in range(-(-n // PAGE), self.table.shape[1]):
                if self.table[b, j] >= 0:
                    self.refs[self.table[b, j]] -= 1
                    self.table[b, j] = -1

    def compact(self):
        used = self.refs > 0
        U = int(used.sum())
        N = len(used)
        new_id = np.where(used, np.arange(N), -1).astype(np.int32)
        holes = [p for p in range(U) if not used[p]]
        movers = [p for p in range(N - 1, U - 1, -1) if used[p]]
        for h, m in zip(holes, movers):
            self.kv[h], self.idx[h] = self.kv[m], self.idx[m]
            self.refs[h], self.refs[m] = self.refs[m], 0
            new_id[m] = h
        self.table = np.where(self.table >= 0, new_id[np.maximum(self.table, 0)], -1).astype(np.int32)
        return new_id, U


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """Device pools and tables with their model; every call is made on both."""

    def __init__(self, seed, B, width, num_pages, held, cap=130):
        g = np.random.default_rng(seed)
        table = np.full((B, width), -1, np.int32)
        refs = np.zeros(num_pages, np.int32)
        ids, at = g.permutation(num_pages), 0
        for b, k in enumerate(held):
            table[b, :k] = ids[at:at + k]
            at += k
        refs[ids[:at]] = 1
        kv = g.integers(0, 256, (num_pages, 18432), dtype=np.uint8)
        idx = g.integers(0, 256, (num_pages, 4352), dtype=np.uint8)
        self.m = Model(table, refs, kv, idx)
        self.kv, self.idx = torch.from_numpy(kv).cuda(), torch.from_numpy(idx).cuda()
        self.table, self.refs = torch.from_numpy(table).cuda(), torch.from_numpy(refs).cuda()
        self.cache = csa.make_cache(self.kv, self.idx, self.table, num_pages, 2)
        self.pages = csa.make_pages(self.table, self.refs)
        self.codes = torch.from_numpy(g.integers(0, 256, (B, cap, 512), dtype=np.uint8)).cuda()
        self.scale = torch.from_numpy(g.random((B, cap), dtype=np.float32)).cuda()
        self.window = csa.make_window(self.codes, self.scale, cap)
        self.pending = torch.from_numpy(g.standard_normal((B, 640)).astype(np.float32)).cuda().bfloat16()
        self.ws = torch.zeros(max(csa.csa_workspace_size(csa.OP_PAGES_RESERVE, 4 * B + 8, width * PAGE, 0),
                                  csa.csa_workspace_size(csa.OP_PAGES_COMPACT, num_pages, 0, 0)),
                              dtype=torch.uint8, device="cuda")
        self.ws[256:] = 0xA5

    def reserve(self, req, first, count, flags=0):
        csa.csa_pages_reserve(self.cache, self.pages, ints(req), ints(first), ints(count), max(count + [0]), self.ws)
        want = self.m.reserve(req, first, count)
        self.check(want | flags)

    def fork(self, parent, child, entries):
        codes, scale, pend = self.codes.clone(), self.scale.clone(), self.pending.clone()
        csa.csa_pages_fork(self.cache, self.pages, self.window, self.pending, ints(parent), ints(child), ints(entries),
                           self.ws)
        self.m.fork(parent, child, entries)
        for p, c in zip(parent, child):
            if c >= 0:
                codes[c], scale[c], pend[c] = codes[p], scale[p], pend[p]
        assert torch.equal(codes, self.codes) and torch.equal(scale, self.scale)
        assert torch.equal(pend.view(torch.int16), self.pending.view(torch.int16))
        self.check(0)

    def free(self, req, keep=None):
        csa.csa_pages_free(self.cache, self.pages, ints(req), None if keep is None else ints(keep), self.ws)
        self.m.free(req, keep or [0] * len(req))
        self.check(0)

    def compact(self, outputs=True):
        N = len(self.m.refs)
        new_id, used = torch.full((N,), 77, dtype=torch.int32, device="cuda"), ints([77])
        csa.csa_pages_compact(self.cache, self.pages, new_id if outputs else None, used if outputs else None, self.ws)
        want, U = self.m.compact()
        if outputs:
            assert np.array_equal(new_id.cpu().numpy(), want) and int(used) == U
        self.check(0)

    def check(self, flags):
        assert csa.csa_check_device_status(self.ws) == ((5, flags) if flags else (0, 0))
        assert np.array_equal(self.table.cpu().numpy(), self.m.table), "page table"
        assert np.array_equal(self.refs.cpu().numpy(), self.m.refs), "counts"
        assert np.array_equal(self.kv.cpu().numpy(), self.m.kv), "main-KV pool"
        assert np.array_equal(self.idx.cpu().numpy(), self.m.idx), "indexer pool"


# ---- each call ------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("num_pages", [5, 64, 515, 4100])
def test_reserve_takes_the_lowest_free_pages_in_order(num_pages):
    held = [min(num_pages // 4, 3), 1, 0]
    p = Pool(num_pages, 3, 9, num_pages, held)
    first = [64 * held[0] - 5, 0, 0]
    p.reserve([0, 1, 2], [max(0, f) for f in first], [1, 64, 65])
    p.reserve([0, 1, 2], [max(0, f) + 1 for f in first], [1, 1, 1])      # all of them held already
    p.reserve([1, 2, -1, -1], [200, 0, 9, 9], [0, 1, 9, 9])              # nothing asked, padding


@gpu
def test_reserve_runs_out_of_pages():
    p = Pool(7, 3, 40, 20, [4, 3, 2])
    p.reserve([0, 1, 2], [256, 192, 128], [300, 900, 64], flags=csa.FLAG_NO_PAGES)
    p.reserve([0], [2000], [1], flags=csa.FLAG_NO_PAGES)
    p.reserve([0], [0], [1])


@gpu
@pytest.mark.parametrize("entries", [0, 1, 63, 64, 65, 300])
def test_fork_shares_and_reserve_copies_on_write(entries):
    p = Pool(11 + entries, 6, 9, 40, [6, 5, 0, 0, 3, 0])
    p.fork([0, 0, 1, 1], [2, 3, 4, 5], [entries, entries, min(entries, 300), 64])   # 4 gives up its own pages
    p.reserve([0, 2, 3, 4, 5], [entries] * 5, [2, 2, 1, 0, 1])
    p.reserve([0, 2, 3, 4, 5], [entries] * 5, [2, 2, 1, 70, 1])


@gpu
def test_every_holder_copies_at_once_frees_the_page():
    p = Pool(21, 2, 4, 8, [1, 0])
    p.fork([0], [1], [10])
    shared = int(p.table[0, 0])
    p.reserve([0, 1], [10, 10], [1, 1])
    assert int(p.refs[shared]) == 0
    p.reserve([0, 1], [64, 64], [1, 1])


@gpu
def test_fork_again_replaces_what_the_child_shared():
    p = Pool(23, 4, 6, 30, [5, 4, 0, 0])
    p.fork([0, 0], [2, 3], [320, 320])
    p.fork([0, 1], [2, 3], [100, 256])
    p.fork([2], [3], [64])


@gpu
def test_free_keeps_a_prefix_and_releases_the_rest():
    p = Pool(31, 5, 9, 60, [9, 7, 5, 3, 0])
    p.fork([0], [4], [500])
    p.free([0, 1, 2, 3, 4], [65, 64, 0, 1000, 1])
    p.free([0, 2, 4, -1], None)
    p.free([1, 3])


@gpu
@pytest.mark.parametrize("num_pages,held", [(1, [0]), (1, [1]), (7, [3, 2]), (64, [0, 0]), (64, [40, 24]), (333, [5, 100, 3]),
                                            (5000, [700, 1, 900, 33])])
def test_compact_moves_the_highest_pages_into_the_lowest_holes(num_pages, held):
    p = Pool(41 + num_pages, len(held) + 1, max(held) + 1, num_pages, held + [0])
    if held[0] > 1:
        p.fork([0], [len(held)], [64 * (held[0] - 1)])
    p.compact()
    p.compact(outputs=False)                    # nothing left to move
    if held[0] > 2:
        p.free([0], [64])
        p.compact(outputs=False)


@gpu
def test_compact_keeps_a_page_held_outside_the_table():
    p = Pool(47, 1, 3, 20, [2])
    free = int(np.nonzero(p.m.refs == 0)[0][-1])
    p.refs[free] = 1
    p.m.refs[free] = 1
    p.compact()


# ---- faults that only the device sees ---------------------------------------------------
@gpu
@pytest.mark.parametrize("req", [[0, 0], [1, 0], [0, 4], [-1, 2], [0, -1, 2]])
def test_bad_lists_change_nothing(req):
    p = Pool(51, 4, 6, 40, [3, 2, 1, 0])
    n = len(req)
    f = csa.FLAG_ROW_INVALID
    csa.csa_pages_reserve(p.cache, p.pages, ints(req), ints([0] * n), ints([300] * n), 300, p.ws)
    p.check(f)
    csa.csa_pages_free(p.cache, p.pages, ints(req), None, p.ws)
    p.check(f)
    before = p.codes.clone()
    csa.csa_pages_fork(p.cache, p.pages, p.window, p.pending, ints([3] * n), ints(req), ints([64] * n), p.ws)
    p.check(f)
    for parent in (-1, 4, 1, 0):                # out of range, or itself a child
        csa.csa_pages_fork(p.cache, p.pages, p.window, p.pending, ints([3, parent]), ints([0, 1]), ints([0, 0]), p.ws)
        p.check(f)
    assert torch.equal(before, p.codes)


@gpu
def test_bad_units_are_left_out():
    p = Pool(53, 4, 6, 40, [3, 2, 1, 0])
    lists = [([-1, 0, 0, 0], [64, 0, 0, 0]), ([0, 0, 0, 384], [1, -1, 9, 1]), ([2 ** 31 - 1, 0, 0, 0], [64, 0, 0, 0])]
    for first, count in lists:
        csa.csa_pages_reserve(p.cache, p.pages, ints([0, 1, 2, 3]), ints(first), ints(count), 64, p.ws)
        p.check(csa.FLAG_ROW_INVALID)
    csa.csa_pages_reserve(p.cache, p.pages, ints([3]), ints([0]), ints([65]), 64, p.ws)      # past the host's bound
    p.check(csa.FLAG_ROW_INVALID)
    for n in (-1, 385, 2 ** 31 - 1):
        csa.csa_pages_fork(p.cache, p.pages, None, None, ints([0]), ints([3]), ints([n]), p.ws)
        p.check(csa.FLAG_ROW_INVALID)
    csa.csa_pages_free(p.cache, p.pages, ints([0]), ints([-1]), p.ws)
    p.check(csa.FLAG_ROW_INVALID)


@gpu
def test_bad_slots_are_flagged():
    oob = csa.FLAG_PAGE_OOB
    p = Pool(57, 3, 4, 30, [3, 2, 0])
    lost = int(np.nonzero(p.m.refs == 0)[0][-1])
    for bad in (30, 2 ** 31 - 1, lost):         # past the pool, or without a count
        p.table[0, 1] = bad
        p.m.table[0, 1] = bad
        csa.csa_pages_reserve(p.cache, p.pages, ints([0]), ints([64]), ints([1]), 1, p.ws)
        p.check(oob)
        csa.csa_pages_fork(p.cache, p.pages, None, None, ints([0]), ints([2]), ints([192]), p.ws)
        p.m.table[2] = [p.m.table[0, 0], -1, p.m.table[0, 2], -1]
        p.m.refs[p.m.table[0, [0, 2]]] += 1
        p.check(oob)
        p.free([2])
        csa.csa_pages_free(p.cache, p.pages, ints([0]), ints([64]), p.ws)
        p.m.refs[p.m.table[0, 2]] -= 1
        p.m.table[0, 1:] = -1
        p.check(oob)
        p.reserve([0], [64], [128])
    p.table[1, 3] = 30
    p.m.table[1, 3] = -1
    csa.csa_pages_compact(p.cache, p.pages, None, None, p.ws)
    p.m.compact()
    p.check(oob)


# ---- together ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_random_runs_of_all_calls(seed):
    g = np.random.default_rng(seed)
    B, width = 12, 10
    p = Pool(100 + seed, B, width, 150, [int(x) for x in g.integers(0, 7, B)])
    for _ in range(12):
        some = sorted(int(x) for x in g.choice(B, int(g.integers(1, B)), replace=False))
        what = g.integers(0, 4)
        if what == 0:
            child = some[: len(some) // 2 + 1]
            rest = [b for b in range(B) if b not in child]
            if rest:
                p.fork([int(g.choice(rest)) for _ in child], child, [int(g.integers(0, width * PAGE + 1)) for _ in child])
        elif what == 1:
            first = [int(g.integers(0, width * PAGE - 200)) for _ in some]
            p.reserve(some, first, [int(g.integers(0, 200)) for _ in some])
        elif what == 2:
            p.free(some, [int(g.integers(0, width * PAGE)) for _ in some])
        else:
            p.compact()


@gpu
def test_captured_step_reserves_appends_and_attends():
    """A step of reserve, append and dense attention in one graph, replayed while
    the requests grow over page borders after a fork, equals the same step on
    requests that own all their pages from the start."""
    from fp4_sparse_attention_csa_gb300 import workloads as W
    from fp4_sparse_attention_csa_gb300.session import DeviceState

    steps, H = 5, 16
    ctx = [253, 380]                            # P = 2: entries 126 and 190 (the page borders are 128 and 192)
    wl = W.custom("pages", 5, [c + 40 for c in ctx], [40, 40], H=H, Hi=16)

    def run(managed):
        st = DeviceState(wl)
        for b, c in enumerate(ctx):             # the history alone
            x, y = wl.tokens(b, 0, c)
            pos0, off = np.zeros(2, np.int32), np.zeros(3, np.int64)
            off[b + 1:] = c
            st.append(pos0, off, x, y)
        B, maxp = 3, wl.max_pages
        kv = torch.zeros(40, 18432, dtype=torch.uint8, device="cuda")
        idx = torch.zeros(40, 4352, dtype=torch.uint8, device="cuda")
        n = wl.num_pages
        kv[:n], idx[:n] = st.kv_pool.view(n, -1), st.idx_pool.view(n, -1)
        table = torch.full((B, maxp), -1, dtype=torch.int32, device="cuda")
        refs = torch.zeros(40, dtype=torch.int32, device="cuda")
        for b, c in enumerate(ctx):
            k = -(-(c // 2) // PAGE)
            table[b, :k] = st.page_table[b, :k]
            refs[st.page_table[b, :k].long()] = 1
        cap = wl.win_cap
        codes = torch.zeros(B, cap, 512, dtype=torch.uint8, device="cuda")
        scale = torch.zeros(B, cap, device="cuda")
        pend = torch.zeros(B, 640, dtype=torch.bfloat16, device="cuda")
        codes[:2], scale[:2], pend[:2] = st.win_codes.view(2, cap, 512), st.win_scale.view(2, cap), st.pending
        cache, pages = csa.make_cache(kv, idx, table, 40, 2), csa.make_pages(table, refs)
        window = csa.make_window(codes, scale, cap)
        ws = torch.zeros(csa.csa_workspace_size(csa.OP_PAGES_RESERVE, B, 1, 0), dtype=torch.uint8, device="cuda")
        csa.csa_pages_fork(cache, pages, window, pend, ints([0]), ints([2]), ints([ctx[0] // 2]), ws)
        lens = torch.tensor([ctx[0], ctx[1], ctx[0]], dtype=torch.int32, device="cuda")
        req = ints([0, 1, 2])
        if not managed:                         # everything private and present before the first step
            big = torch.zeros(csa.csa_workspace_size(csa.OP_PAGES_RESERVE, B, 400, 0), dtype=torch.uint8, device="cuda")
            csa.csa_pages_reserve(cache, pages, req, ints([0, 0, 0]), lens // 2 + 20, 400, big)
            assert csa.csa_check_device_status(big) == (0, 0)
        g = torch.Generator(device="cuda").manual_seed(1)
        kvin = torch.randn(steps, B, 512, generator=g, device="cuda").bfloat16()
        ixin = torch.randn(steps, B, 128, generator=g, device="cuda").bfloat16()
        qs = torch.randn(steps, B, H, 512, generator=g, device="cuda").bfloat16()
        one, kb, ib, qb = ints([1, 1, 1]), kvin[0].clone(), ixin[0].clone(), qs[0].clone()
        off, rows = ints([0, 1, 2, 3]), csa.make_rows(req, lens, maxp * PAGE, 1)
        out = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, H, device="cuda")
        dws = torch.zeros(csa.csa_workspace_size(csa.OP_DENSE_ATTN, B, maxp * PAGE, H), dtype=torch.uint8, device="cuda")
        first = torch.empty_like(lens)

        def step():
            torch.div(lens, 2, rounding_mode="floor", out=first)
            if managed:
                csa.csa_pages_reserve(cache, pages, req, first, one, 1, ws)
            csa.csa_append(cache, window, lens, off, B, kb, ib, pend, ws)
            csa.csa_dense_attn(cache, window, rows, H, qb, 512 ** -0.5, out, lse, None, dws)
            lens.add_(1)

        start = lens.clone()
        saved = [t.clone() for t in (kv, idx, table, refs, codes, scale, pend)]
        step()                                  # warm, then back to the start
        for t, v in zip((kv, idx, table, refs, codes, scale, pend), saved):
            t.copy_(v)
        lens.copy_(start)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        got = []
        for t in range(steps):
            kb.copy_(kvin[t])
            ib.copy_(ixin[t])
            qb.copy_(qs[t])
            graph.replay()
            got.append((out.clone(), lse.clone()))
        assert csa.csa_check_device_status(ws) == (0, 0) and csa.csa_check_device_status(dws) == (0, 0)
        return got

    for (a, la), (b, lb) in zip(run(True), run(False)):
        assert torch.equal(a, b) and torch.equal(la, lb)
        assert not torch.equal(a[0], a[2])      # the parent and the child attend with their own queries


@gpu
def test_every_child_of_a_slot_without_a_count_finds_it_empty():
    """63 children share a parent one of whose pages has no count: none of them
    takes it for another's, whatever their order."""
    p = Pool(59, 64, 40, 200, [30] + [0] * 63)
    lost = [int(x) for x in np.nonzero(p.m.refs == 0)[0][:10]]
    p.table[0, 30:] = ints(lost)
    table, refs = p.table.clone(), p.refs.clone()
    p.m.table[1:, :30] = p.m.table[0, :30]
    p.m.table[0, 30:] = lost
    p.m.refs[p.m.table[0, :30]] += 63
    for _ in range(30):
        p.table.copy_(table)
        p.refs.copy_(refs)
        csa.csa_pages_fork(p.cache, p.pages, None, None, ints([0] * 63), ints(list(range(1, 64))), ints([40 * 64] * 63),
                           p.ws)
        p.check(csa.FLAG_PAGE_OOB)
