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
