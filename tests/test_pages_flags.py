"""csa_pages_*: every fault of a call is reported, also by a thread that meets
two of them, and a child forked before its parent's end."""
import numpy as np
import pytest
import torch

import fp4_sparse_attention_csa_gb300 as csa
from test_pages import Pool, ints

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


@gpu
@pytest.mark.parametrize("first", [-1, 2 ** 31 - 1])
def test_reserve_reports_a_bad_page_and_a_bad_request_of_one_thread(first):
    """1024 units a request and 16 of them: a thread of the plan takes the same
    unit of two requests, whose faults differ."""
    width = 1030
    p = Pool(71, 16, width, 40, [2] + [0] * 15)
    p.table[0, 0] = 40                                    # past the pool
    p.m.table[0, 0] = 40
    most = 1022 * 64
    ws = torch.zeros(csa.csa_workspace_size(csa.OP_PAGES_RESERVE, 16, most, 0), dtype=torch.uint8, device="cuda")
    csa.csa_pages_reserve(p.cache, p.pages, ints(list(range(16))), ints([0, first] + [0] * 14), ints([1, 64] + [0] * 14),
                          most, ws)
    assert csa.csa_check_device_status(ws) == (5, csa.FLAG_PAGE_OOB | csa.FLAG_ROW_INVALID)
    p.check(0)                                            # nothing was changed


@gpu
@pytest.mark.parametrize("back", [0, 1, 72])
def test_a_child_forked_within_the_ring_attends_like_its_parent(back):
    """The ring holds the parent's last 200 tokens: a child forked up to 200 - 128
    tokens before the parent's end has its last token's whole window."""
    from dense_ref import Case

    n, cap, H = 500, 200, 16
    c = Case(600, [n, 70], 1, cap)
    q = c.queries(1, H)
    pos = n - back - 1
    assert c.run(csa, [0], [pos], H, q) == (0, 0)
    c.check([0], [pos], H, q)
    want, lse = c.out.clone(), c.lse.clone()
    held = c.d_table[c.d_table >= 0].long()
    refs = torch.zeros((c.num_pages + 3) // 4 * 4, dtype=torch.int32, device="cuda")
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    csa.csa_pages_fork(c.cache, csa.make_pages(c.d_table, refs), c.window, None, ints([0]), ints([1]), ints([pos + 1]), c.ws)
    c.d_req.fill_(1)
    c.out.fill_(7.0)
    c.call()
    assert csa.csa_check_device_status(c.ws) == (0, 0)
    assert torch.equal(c.out, want) and torch.equal(c.lse, lse)


@gpu
def test_a_fork_without_window_or_pending_leaves_the_childs_own():
    p = Pool(73, 3, 6, 40, [5, 0, 2])
    codes, scale, pend = p.codes.clone(), p.scale.clone(), p.pending.clone()
    csa.csa_pages_fork(p.cache, p.pages, None, None, ints([0]), ints([1]), ints([100]), p.ws)
    p.m.fork([0], [1], [100])
    p.check(0)
    assert torch.equal(codes, p.codes) and torch.equal(scale, p.scale) and torch.equal(pend, p.pending)
