"""Cases, plain forms and calls of two groups of operators over the 4-bit paged cache:

* dense attention: softmax attention of each query row over every visible
  main-KV entry (512 e2m1 codes, one E4M3 scale per 16) and its FP8 window,
  for one token, a few verify rows and whole prompt chunks;
* page management: forking requests, reserving (allocating, copying on write),
  freeing and compacting pages.

`run` computes the plain form in elementary torch operations, or with `own`
calls the library.
"""
import math

import torch

own = False

D, WIN, PAGE = 512, 128, 64
KV_PAGE, IDX_PAGE = 18432, 4352
LOWEST = -math.inf


# ---- cases --------------------------------------------------------------------------
def listed():
    def attn(name, requests, rows, heads, lo, hi, ratio, rope=False, window=True):
        return {"name": name, "kind": "attn", "requests": requests, "rows": rows, "heads": heads, "lo": lo, "hi": hi,
                "ratio": ratio, "rope": rope, "window": window}

    return [
        # one short request, one token: latency alone
        attn("one token, 4k context", 1, 1, 16, 4096, 4096, 2),
        # one long request at 64 heads: the cache split over the whole GPU
        attn("one token, 32k context", 1, 1, 64, 32768, 32768, 2),
        # speculative verify: anchor and five draft rows per request, odd lengths, rotary tables
        attn("verify 32 x 6 rows", 32, 6, 64, 4099, 6143, 2, rope=True),
        # a serving batch of mixed lengths on shuffled pages
        attn("serving 128 rows", 128, 1, 64, 4096, 131072, 2),
        # the layer that keeps one entry per token, at long context
        attn("unpooled 4 x 262144", 4, 1, 64, 262144, 262144, 1),
        # chunked prefill: 128 new rows per request over its history
        attn("extend 4 x 128 rows", 4, 128, 64, 8320, 16512, 2),
        # whole prompts from their first token, odd length, fewer heads, no window
        attn("prompts 2 x 999 rows", 2, 999, 32, 999, 999, 1, window=False),
        # two beams of a short request continue from one prefix
        {"name": "fork 2 short", "kind": "fork", "requests": 2, "children": 1, "lo": 1000, "hi": 1500, "new": 1},
        # parallel samples of a serving batch: three children each, one more block reserved
        {"name": "fork 64 x 3", "kind": "fork", "requests": 64, "children": 3, "lo": 4096, "hi": 131072, "new": 70},
        # requests end and new prompts take their place
        {"name": "turnover 96 of 192", "kind": "turnover", "requests": 192, "lo": 2048, "hi": 65536, "new": 4000},
        # a small and a large fragmented pool closed up
        {"name": "compact 1500 pages", "kind": "compact", "pages": 1500, "used": 0.4, "requests": 12},
        {"name": "compact 49999 pages", "kind": "compact", "pages": 49999, "used": 0.55, "requests": 100},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attn", "attn", "attn", "fork", "turnover", "compact"])
    if kind == "attn":
        heads = rng.choice([16, 32, 64])
        ratio = rng.choice([1, 2])
        rows = rng.choice([1, 1, log(2, 9), log(10, 300)])
        requests = log(1, 96)
        # bounded by the work of the serving batch
        hi = max(rows, min(200000, int(1.2e12 / (requests * rows * heads * 2048 * 2) * ratio)))
        b = max(rows, log(max(rows, 33), max(hi, rows, 34)))
        return {"kind": kind, "requests": requests, "rows": rows, "heads": heads, "lo": max(rows, b // rng.choice([1, 2, 3])),
                "hi": b, "ratio": ratio, "rope": rng.random() < 0.3, "window": rng.random() < 0.7}
    if kind == "fork":
        hi = log(200, 60000)
        return {"kind": kind, "requests": log(1, 64), "children": rng.choice([1, 2, 3]), "lo": max(1, hi // 3), "hi": hi,
                "new": log(1, 300)}
    if kind == "turnover":
        hi = log(200, 60000)
        return {"kind": kind, "requests": log(2, 190), "lo": max(1, hi // 5), "hi": hi, "new": log(1, 8000)}
    return {"kind": kind, "pages": log(300, 45000), "used": round(rng.uniform(0.05, 0.95), 3), "requests": log(1, 100)}


def lengths(n, lo, hi):
    """n context lengths spread evenly over the logarithm of [lo, hi], in a fixed mixed order."""
    span = [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]
    step = next(s for s in (7, 11, 13, 5, 3, 1) if math.gcd(s, n) == 1)
    return [span[i * step % n] for i in range(n)]


# ---- inputs -------------------------------------------------------------------------
def fill_entries(kv, gen):
    """Every entry of the pages: N(0, 1) latents, one in 16 scaled by 4 (salient positions), in NVFP4."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=kv.device)
    for p in range(0, kv.shape[0], 1024):
        n = min(1024, kv.shape[0] - p)
        x = torch.randn(n * PAGE, 32, 16, generator=gen, device=kv.device)
        x *= 1 + 3 * (torch.rand(n * PAGE, 1, 1, generator=gen, device=kv.device) < 1 / 16)
        s8 = (x.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn)
        y = x / s8.float().clamp_min(2.0 ** -9)
        code = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
        code = code.view(n, PAGE * 256, 2)
        kv[p:p + n, :16384] = code[..., 0] | (code[..., 1] << 4)
        kv[p:p + n, 16384:] = s8.view(torch.uint8).view(n, PAGE * 32)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    return (prepare_attn if case["kind"] == "attn" else prepare_pages)(case, gen, dev)


def prepare_attn(case, gen, dev):
    B, r, H, P = case["requests"], case["rows"], case["heads"], case["ratio"]
    ctx = torch.tensor(lengths(B, case["lo"], case["hi"]))
    pages = [max(1, -(-(int(c) // P) // PAGE)) for c in ctx]
    n, width = sum(pages), max(pages)
    kv = torch.empty(n, KV_PAGE, dtype=torch.uint8, device=dev)
    fill_entries(kv, gen)
    ids = torch.randperm(n, generator=gen, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = ids[at:at + k]
        at += k
    cap = WIN + r - 1
    tok = torch.randn(B * cap, D, generator=gen, device=dev)
    scale = tok.abs().amax(-1) / 448
    th = torch.rand(int(ctx.max()), 32, generator=gen, device=dev) * (2 * math.pi)
    s = {
        "case": case, "kv": kv, "idx": torch.zeros(n, IDX_PAGE, dtype=torch.uint8, device=dev), "table": table,
        "codes": (tok / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), "wscale": scale, "cap": cap,
        "cos": torch.cos(th), "sin": torch.sin(th),
        "req": torch.arange(B, device=dev).repeat_interleave(r).int(),
        "pos": (ctx[:, None] - r + torch.arange(r)).reshape(-1).int().to(dev),
        "q": torch.randn(B * r, H, D, generator=gen, device=dev).bfloat16(), "scale": 1 / math.sqrt(D),
        "entries": max(int(c) // P for c in ctx),
        "out": torch.empty(B * r, H, D, dtype=torch.bfloat16, device=dev),
        "lse": torch.empty(B * r, H, dtype=torch.float32, device=dev),
    }
    if own:  # what a serving program sets up once for its cache and its step
        import fp4_sparse_attention_csa_gb300 as csa
        s["cache"] = csa.make_cache(kv, s["idx"], table, n, P)
        s["window"] = csa.make_window(s["codes"], scale, cap) if case["window"] else None
        s["rows"] = csa.make_rows(s["req"], s["pos"], s["entries"], r)
        s["opts"] = csa.make_opts(rope_cos=s["cos"], rope_sin=s["sin"]) if case["rope"] else None
        s["ws"] = torch.zeros(csa.csa_workspace_size(csa.OP_DENSE_ATTN, B * r, s["entries"], H), dtype=torch.uint8,
                              device=dev)
    return s


def pages_of(case):
    """(entries of each request slot, pages of the pool) of a page case."""
    if case["kind"] == "fork":
        ent = lengths(case["requests"], case["lo"], case["hi"])
        ent = ent + [0] * (case["requests"] * case["children"])
        more = len(ent) * (case["new"] // PAGE + 2)
    elif case["kind"] == "turnover":
        ent = lengths(case["requests"], case["lo"], case["hi"])
        more = len(ent) * (case["new"] // PAGE + 2)
    else:
        used = max(case["requests"], int(case["pages"] * case["used"]))
        each = [used // case["requests"] + (i < used % case["requests"]) for i in range(case["requests"])]
        return [PAGE * k - (7 * i + 3) % PAGE for i, k in enumerate(each)], max(used, case["pages"])
    used = sum(-(-e // PAGE) for e in ent)
    return ent, used + used // 4 + more


def prepare_pages(case, gen, dev):
    ent, n = pages_of(case)
    held = [-(-e // PAGE) for e in ent]
    width = max(held) + case.get("new", 0) // PAGE + 2
    table = torch.full((len(ent), width), -1, dtype=torch.int32, device=dev)
    ids = torch.randperm(n, generator=gen, device=dev).int()  # used pages lie all over the pool
    refs = torch.zeros(n, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = ids[at:at + k]
        at += k
    refs[ids[:at].long()] = 1
    share = case["kind"] == "compact" and len(ent) > 1
    if share:  # the second request continues from the first's leading pages
        k = min(held[0], held[1]) // 2
        if k:
            refs[table[1, :k].long()] -= 1
            table[1, :k] = table[0, :k]
            refs[table[0, :k].long()] += 1
    B, cap = len(ent), 256
    s = {"case": case, "kv": torch.randint(0, 256, (n, KV_PAGE), generator=gen, device=dev, dtype=torch.uint8),
         "idx": torch.randint(0, 256, (n, IDX_PAGE), generator=gen, device=dev, dtype=torch.uint8),
         "table0": table, "refs0": refs, "table": table.clone(), "refs": refs.clone(),
         "new_id": torch.empty(n, dtype=torch.int32, device=dev), "num_used": torch.empty(1, dtype=torch.int32, device=dev)}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if case["kind"] == "fork":
        nb, c = case["requests"], case["children"]
        s["codes"] = torch.randint(0, 256, (B * cap, D), generator=gen, device=dev, dtype=torch.uint8)
        s["wscale"] = torch.rand(B * cap, generator=gen, device=dev)
        s["pending"] = torch.randn(B, 640, generator=gen, device=dev).bfloat16()
        s["parent"] = ints([i // c for i in range(nb * c)])
        s["child"] = ints([nb + i for i in range(nb * c)])
        s["share"] = ints([ent[i // c] for i in range(nb * c)])
        s["req"], s["first"] = ints(list(range(B))), ints(ent[:nb] + [ent[i // c] for i in range(nb * c)])
        s["count"] = ints([case["new"]] * B)
    elif case["kind"] == "turnover":
        s["req"] = ints(list(range(0, B, 2)))
        s["keep"], s["first"] = ints([0] * len(range(0, B, 2))), ints([0] * len(range(0, B, 2)))
        s["count"] = ints([max(1, case["new"] - 13 * (i % 5)) for i in range(0, B, 2)])
    if own:
        import fp4_sparse_attention_csa_gb300 as csa
        s["cache"] = csa.make_cache(s["kv"], s["idx"], s["table"], n, 2)
        s["pages"] = csa.make_pages(s["table"], s["refs"])
        s["window"] = csa.make_window(s["codes"], s["wscale"], cap) if "codes" in s else None
        size = max(csa.csa_workspace_size(csa.OP_PAGES_RESERVE, B, case.get("new", 0), 0),
                   csa.csa_workspace_size(csa.OP_PAGES_COMPACT, n, 0, 0))
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device=dev)
    return s


# ---- one pass -----------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["kind"] == "attn":
        if own:
            import fp4_sparse_attention_csa_gb300 as csa
            csa.csa_dense_attn(s["cache"], s["window"], s["rows"], case["heads"], s["q"], s["scale"], s["out"], s["lse"],
                               s["opts"], s["ws"])
            return s["out"], s["lse"]
        return plain_attn(s)
    # the bookkeeping starts from the same tables in each pass
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if own:
        import fp4_sparse_attention_csa_gb300 as csa
        if case["kind"] == "fork":
            csa.csa_pages_fork(s["cache"], s["pages"], s["window"], s["pending"], s["parent"], s["child"], s["share"], s["ws"])
            csa.csa_pages_reserve(s["cache"], s["pages"], s["req"], s["first"], s["count"], case["new"], s["ws"])
        elif case["kind"] == "turnover":
            csa.csa_pages_free(s["cache"], s["pages"], s["req"], s["keep"], s["ws"])
            csa.csa_pages_reserve(s["cache"], s["pages"], s["req"], s["first"], s["count"], case["new"], s["ws"])
        else:
            csa.csa_pages_compact(s["cache"], s["pages"], s["new_id"], s["num_used"], s["ws"])
    elif case["kind"] == "fork":
        plain_fork(s)
        plain_reserve(s, case["new"])
    elif case["kind"] == "turnover":
        plain_free(s)
        plain_reserve(s, case["new"])
    else:
        plain_compact(s)
    if case["kind"] == "fork":
        # copies: compared bit for bit
        return (s["table"], s["refs"], s["kv"], s["idx"], s["codes"], s["wscale"].view(torch.int32),
                s["pending"].view(torch.int16))
    if case["kind"] == "turnover":
        return s["table"], s["refs"]
    return s["table"], s["refs"], s["kv"], s["idx"], s["new_id"], s["num_used"]


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = E2M1 + [-v for v in E2M1]


def rotate(x, cos, sin):
    """Rotate-half on the last 64 dims."""
    a, b = x[..., 448:480], x[..., 480:]
    return torch.cat([x[..., :448], a * cos - b * sin, b * cos + a * sin], -1)


def plain_attn(s):
    case = s["case"]
    B, r, H, E = case["requests"], case["rows"], case["heads"], s["entries"]
    pair = torch.tensor([[E2M1[c & 15], E2M1[c >> 4]] for c in range(256)], device=s["kv"].device)
    pages = s["kv"][s["table"].long().clamp_min(0)]                          # [B, pages, bytes]
    keys = pair[pages[..., :16384].int()].view(B, -1, 32, 16)
    keys *= pages[..., 16384:].contiguous().view(torch.float8_e4m3fn).float().view(B, -1, 32, 1)
    keys = keys.view(B, -1, D)[:, :E]
    pos = s["pos"].view(B, r).long()
    q = s["q"].float().view(B, r, H, D)
    if case["rope"]:
        q = rotate(q, s["cos"][pos][:, :, None], s["sin"][pos][:, :, None])
    seen = torch.arange(keys.shape[1], device=pos.device) < ((pos + 1) // case["ratio"])[..., None]
    logit = torch.bmm(q.reshape(B, r * H, D), keys.transpose(1, 2)).view(B, r, H, -1) * s["scale"]
    logit.masked_fill_(~seen[:, :, None], LOWEST)
    if case["window"]:
        at = (pos - (WIN - 1)).clamp_min(0)[..., None] + torch.arange(WIN, device=pos.device)   # [B, r, 128]
        slot = torch.arange(B, device=pos.device)[:, None, None] * s["cap"] + at % s["cap"]
        near = s["codes"][slot].view(torch.float8_e4m3fn).float() * s["wscale"][slot][..., None]
        if case["rope"]:
            p = torch.minimum(at, pos[..., None])
            near = rotate(near, s["cos"][p], s["sin"][p])
        wlog = torch.matmul(q, near.transpose(-1, -2)) * s["scale"]
        wlog.masked_fill_((at > pos[..., None])[:, :, None], LOWEST)
        logit = torch.cat([logit, wlog], -1)
    m = logit.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(logit - m)
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p[..., :keys.shape[1]].reshape(B, r * H, -1), keys).view(B, r, H, D)
    if case["window"]:
        o = o + torch.matmul(p[..., keys.shape[1]:], near)
    out = torch.where(l > 0, o / l, torch.zeros_like(o)).bfloat16()
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, LOWEST))
    return out.view(B * r, H, D), lse.view(B * r, H)


def held_once(table, req):
    """One per slot of these requests' rows that names a page, and the pages."""
    rows = table[req]
    return (rows >= 0).int().view(-1), rows.clamp_min(0).view(-1).long()


def plain_fork(s):
    table, refs = s["table"], s["refs"]
    parent, child = s["parent"].long(), s["child"].long()
    had, page = held_once(table, child)
    refs.index_add_(0, page, -had)
    slot = torch.arange(table.shape[1], device=table.device)
    table[child] = torch.where(slot < ((s["share"] + PAGE - 1) // PAGE)[:, None], table[parent], -1)
    has, page = held_once(table, child)
    refs.index_add_(0, page, has)
    B = table.shape[0]
    for name in ("codes", "wscale", "pending"):
        ring = s[name].view(B, -1)
        ring[child] = ring[parent]


def plain_free(s):
    table, refs, req = s["table"], s["refs"], s["req"].long()
    slot = torch.arange(table.shape[1], device=table.device)
    drop = slot >= ((s["keep"] + PAGE - 1) // PAGE)[:, None]
    rows = table[req]
    refs.index_add_(0, rows.clamp_min(0).view(-1).long(), -(drop & (rows >= 0)).int().view(-1))
    table[req] = torch.where(drop, -1, rows)


def plain_reserve(s, most):
    table, refs, req = s["table"], s["refs"], s["req"].long()
    first, count = s["first"].long(), s["count"].long()
    lp = (first // PAGE)[:, None] + torch.arange(most // PAGE + 2, device=table.device)
    wanted = (count > 0)[:, None] & (lp <= ((first + count - 1) // PAGE)[:, None])
    lp = lp.clamp_max(table.shape[1] - 1)
    page = table[req[:, None], lp]
    shared = (page >= 0) & (refs[page.clamp_min(0).long()] > 1)
    need = wanted & ((page < 0) | shared)
    free = torch.nonzero(refs <= 0).view(-1)                              # lowest first
    unit = torch.nonzero(need.view(-1)).view(-1)[:free.numel()]
    new = free[:unit.numel()]
    old = page.view(-1)[unit].long()
    copy = old >= 0
    s["kv"][new[copy]] = s["kv"][old[copy]]
    s["idx"][new[copy]] = s["idx"][old[copy]]
    refs.index_add_(0, old[copy], torch.full_like(old[copy], -1, dtype=torch.int32))
    refs[new] = 1
    table[req[:, None].expand_as(lp).reshape(-1)[unit], lp.reshape(-1)[unit]] = new.int()


def plain_compact(s):
    table, refs = s["table"], s["refs"]
    place = torch.arange(refs.numel(), device=refs.device)
    used = refs > 0
    total = used.sum()
    hole = torch.nonzero(~used & (place < total)).view(-1)
    mover = torch.nonzero(used & (place >= total)).view(-1).flip(0)      # the highest goes to the lowest hole
    new_id = torch.where(used, place, -1)
    new_id[mover] = hole
    s["kv"][hole] = s["kv"][mover]
    s["idx"][hole] = s["idx"][mover]
    refs[hole] = refs[mover]
    refs[mover] = 0
    table.copy_(torch.where(table >= 0, new_id[table.clamp_min(0).long()], -1))
    s["new_id"].copy_(new_id)
    s["num_used"].copy_(total)


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    if case["kind"] == "attn":
        B, r, H, P = case["requests"], case["rows"], case["heads"], case["ratio"]
        ctx = lengths(B, case["lo"], case["hi"])
        pairs = sum((p + 1) // P + (min(p + 1, WIN) if case["window"] else 0) for c in ctx for p in range(c - r, c))
        entries = sum(c // P for c in ctx)
        near = sum(min(c, WIN + r - 1) for c in ctx) if case["window"] else 0
        return {"bytes": entries * 288 + near * 516 + B * r * H * (D * 4 + 4) + entries // PAGE * 4,
                "flops": pairs * H * D * 4}
    ent, n = pages_of(case)
    one = 2 * (KV_PAGE + IDX_PAGE)
    if case["kind"] == "fork":
        kids = case["requests"] * case["children"]
        held = [-(-e // PAGE) for e in ent[:case["requests"]]]
        copied = sum(1 + case["children"] for e in ent[:case["requests"]] if e % PAGE)
        b = copied * one + kids * 2 * (256 * (D + 4) + 1280) + 12 * sum(held) * case["children"] + 4 * n
    elif case["kind"] == "turnover":
        freed = [-(-e // PAGE) for e in ent[::2]]
        b = 4 * n + 12 * sum(freed) + 12 * len(freed) * (case["new"] // PAGE + 1)
    else:
        used = sum(-(-e // PAGE) for e in ent)
        b = int(used * (1 - used / n)) * one + 12 * n
    return {"bytes": b, "flops": 0}


# ---- the definition in 64 bits ------------------------------------------------------
def exact(case, seed):
    """Attention request by request, a key's value from its code's sign, exponent and fraction bits."""
    if case["kind"] != "attn":
        return None
    s = prepare(case, seed)
    B, r, H, P = case["requests"], case["rows"], case["heads"], case["ratio"]
    f64 = torch.float64

    def e4m3(b):
        b = b.long()
        e, m = (b >> 3) & 15, (b & 7).to(f64)
        v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).to(f64)), m * 2.0 ** -9)
        return torch.where(b > 127, -v, v)

    def e2m1(c):
        e, m = (c >> 1) & 3, (c & 1).to(f64)
        v = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).to(f64)), m / 2)
        return torch.where(c > 7, -v, v)

    def turned(x, p):
        a, b = x[..., 448:480].clone(), x[..., 480:].clone()
        c, t = s["cos"].to(f64)[p], s["sin"].to(f64)[p]
        x[..., 448:480], x[..., 480:] = a * c - b * t, b * c + a * t
        return x

    out = torch.zeros(B * r, H, D, dtype=f64, device="cuda")
    lse = torch.full((B * r, H), -math.inf, dtype=f64, device="cuda")
    for b in range(B):
        pos = s["pos"][b * r:(b + 1) * r].long()
        n = (int(pos[-1]) + 1) // P
        raw = s["kv"][s["table"][b, :-(-n // PAGE)].long()]
        code = raw[:, :16384].reshape(-1, 256).long()
        keys = torch.stack([e2m1(code & 15), e2m1(code >> 4)], -1).view(-1, 32, 16)
        keys = (keys * e4m3(raw[:, 16384:].reshape(-1, 32))[..., None]).view(-1, D)[:n]
        wpos = torch.arange(max(0, int(pos[0]) - 127), int(pos[-1]) + 1, device="cuda")
        if case["window"]:
            slot = b * s["cap"] + wpos % s["cap"]
            near = e4m3(s["codes"][slot]) * s["wscale"][slot].to(f64)[:, None]
            near = turned(near, wpos) if case["rope"] else near
        else:
            near, wpos = torch.zeros(0, D, dtype=f64, device="cuda"), wpos[:0]
        every = torch.cat([keys, near])
        for lo in range(0, r, 64):
            row = slice(b * r + lo, b * r + min(r, lo + 64))
            p = pos[lo:lo + 64, None]
            q = s["q"][row].to(f64)
            q = turned(q, p.expand(-1, H)) if case["rope"] else q
            see = torch.cat([torch.arange(n, device="cuda") < (p + 1) // P, (wpos <= p) & (wpos > p - WIN)], 1)
            w = (q.reshape(-1, D) @ every.T).view(-1, H, every.shape[0]) * s["scale"]
            w = w.masked_fill(~see[:, None], -math.inf)
            some = see.any(1)
            if not bool(some.any()):
                continue
            z = torch.logsumexp(w[some], -1)
            at = torch.arange(row.start, row.stop, device="cuda")[some]
            lse[at] = z
            out[at] = (torch.exp(w[some] - z[..., None]).view(-1, every.shape[0]) @ every).view(-1, H, D)
    return out, lse
