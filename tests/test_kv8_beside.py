"""The 8-bit cache beside the latent one, as a model with both kinds of layers uses them: pages reserved for
both, tokens appended to both, rows that attend in both; one page table where an entry is a token, two where an
entry pools two."""
import numpy as np
import pytest
import torch

import dense_ref
import fp4_sparse_attention_csa_gb300 as csa
from kv8_ref import Cache, Device, bf16, dev

gpu = pytest.mark.gpu
H, KV, D = 16, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa.build.build()
    if torch.cuda.is_available():
        torch.cuda.set_device(0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("P", [1, 2])
def test_both_caches_step_by_step(P):
    """Prompts, then tokens; before the last ones request 1 becomes a continuation of request 0 (its pages shared, its
    tail copied) and both go on inside the same page."""
    ctx, steps, pages = [150, 90], 6, 24
    c = Cache(7 + P, [c + steps for c in ctx], KV, D, width=4)
    s = Device(csa, c, filled=False)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    kv, idx = (torch.zeros(pages, n, dtype=torch.uint8, device="cuda") for n in (18432, 4352))
    latent, book = csa.make_cache(kv, idx, table, pages, P), csa.make_pages(table, refs)
    codes, scale = torch.zeros(2, 192, 512, dtype=torch.uint8, device="cuda"), torch.zeros(2, 192, device="cuda")
    window, pend = csa.make_window(codes, scale, 192), torch.zeros(2, 640, dtype=torch.bfloat16, device="cuda")
    if P == 1:                                             # a page is 64 tokens in both: the same table
        s.table, c.pages = table, pages
        s.pool = torch.zeros(pages, KV, csa.kv8_record_bytes(D), dtype=torch.uint8, device="cuda")
        s.codes, s.scale = torch.zeros(pages, KV, D, dtype=torch.int8, device="cuda"), torch.zeros(pages, KV, device="cuda")
        s.cache = csa.make_kv8(s.pool, s.tail, table, pages, KV, D, s.codes, s.scale)
    ws = torch.zeros(max(csa.csa_workspace_size(csa.OP_PAGES_RESERVE, 2, 200, 0), 256), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(P)
    req = ints([0, 1])

    def append(pos0, counts):
        total = sum(counts)
        off, at = ints([0, counts[0], total]), ints(pos0)
        csa.csa_pages_reserve(latent, book, req, at // P, ints([(p + n) // P - p // P for p, n in zip(pos0, counts)]), 200, ws)
        csa.csa_append(latent, window, at, off, total, torch.randn(total, 512, generator=g, device="cuda").bfloat16(),
                       torch.randn(total, 128, generator=g, device="cuda").bfloat16(), pend, ws)
        s.append(pos0, counts)
        assert s.status() == (0, 0)

    def attend(pos):
        at, most = ints(pos), max(pos) + 1
        rows = csa.make_rows(req, at, -(-most // P), 1)
        rows8 = rows if P == 1 else csa.make_rows(req, at, most, 1)   # this cache's bound is in tokens
        q, q8 = bf16(c.rng.standard_normal((2, H, 512))), bf16(c.rng.standard_normal((2, H, D)))
        out, lse = torch.empty(2, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, H, device="cuda")
        out8, lse8 = torch.empty(2, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, H, device="cuda")
        dws = torch.zeros(csa.csa_workspace_size(csa.OP_DENSE_ATTN, 2, rows.max_entries, H), dtype=torch.uint8, device="cuda")
        ws8 = torch.zeros(csa.csa_workspace_size(csa.OP_KV8_ATTN, 2, rows8.max_entries, H), dtype=torch.uint8, device="cuda")
        q_t, q8_t = dev(q, torch.bfloat16), dev(q8, torch.bfloat16)
        csa.csa_dense_attn(latent, window, rows, H, q_t, 512 ** -0.5, out, lse, None, dws)
        csa.csa_kv8_attn(s.cache, rows8, H, q8_t, None, D ** -0.5, out8, lse8, ws8)
        assert csa.csa_check_device_status(dws) == (0, 0) and csa.csa_check_device_status(ws8) == (0, 0)
        t = table.cpu().numpy()
        for b in range(2):
            o, z, do, dz = dense_ref.row_reference(kv.cpu().numpy(), t[b], pages, P, pos[b], q[b], 512 ** -0.5,
                                                   (codes[b].cpu().numpy(), scale[b].cpu().numpy()))
            assert (np.abs(out[b].float().cpu().numpy() - o) <= do).all()
        s.check([0, 1], pos, q8, out8.float().cpu().numpy(), lse8.cpu().numpy())
        if P == 2:                                         # the latent's bound leaves out what lies past it
            csa.csa_kv8_attn(s.cache, rows, H, q8_t, None, D ** -0.5, out8, lse8, ws8)
            assert csa.csa_check_device_status(ws8)[1] == csa.FLAG_ROW_INVALID and not out8[0].any()

    append([0, 0], ctx)
    attend([c - 1 for c in ctx])
    for t in range(3):
        append([c + t for c in ctx], [1, 1])
        attend([c + t for c in ctx])
    # request 1 continues request 0
    n = ctx[0] + 3
    if P == 1:
        csa.csa_pages_fork(latent, book, window, pend, ints([0]), ints([1]), ints([n]), ws)
        s.tail[1] = s.tail[0]
        for k in range(2):
            c.tokens[1] = (c.tokens[0][0].copy(), c.tokens[0][1].copy())
            for x in c.tokens[1]:
                x[n:] = bf16(c.rng.standard_normal(x[n:].shape))
        for t in range(3):
            append([n + t, n + t], [1, 1])
            attend([n + t, n + t])
        assert csa.csa_check_device_status(ws) == (0, 0)
        # every page holds what its request's own tokens give
        c.ctx, c.table = [n + 3, n + 3], table.cpu().numpy()
        want, got = c.fill()[0], s.pool.cpu().numpy()
        used = np.unique(c.table[c.table >= 0])
        assert np.array_equal(got[used], want[used]) and c.table[0, 2] != c.table[1, 2] and c.table[0, 0] == c.table[1, 0]
