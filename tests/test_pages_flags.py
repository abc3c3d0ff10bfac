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
