"""Cases, plain forms and calls of the operators of the 8-bit paged cache of keys and values:

* append: new tokens' keys (rotated on the way) and values into pages of 64 tokens, E4M3 codes with
  one scale per page, head and side, and an int8 summary of each page's keys;
* attn: softmax attention over every token that a row sees;
* select: for each row and key head, the pages that a cheap score on the summaries puts first;
* blocks: softmax attention over the selected pages alone.

`run` computes the plain form in elementary torch operations, or with `own` calls the library.
"""
import math

import torch

own = False

BLOCK, RING = 64, 128
LOWEST = -math.inf
E4M3, F64 = torch.float8_e4m3fn, torch.float64


# ---- cases --------------------------------------------------------------------------
def listed():
    def append(name, requests, new, lo, hi, kv_heads, dim, turn):
        return {"name": name, "kind": "append", "requests": requests, "new": new, "lo": lo, "hi": hi,
                "kv_heads": kv_heads, "dim": dim, "turn": turn}

    def read(kind, name, requests, rows, heads, kv_heads, dim, lo, hi, turn=0, blocks=0):
        return {"name": name, "kind": kind, "requests": requests, "rows": rows, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "lo": lo, "hi": hi, "turn": turn, "blocks": blocks}

    return [
        # a chat's next token: one call of a few microseconds
        append("append one token", 1, 1, 4070, 4070, 8, 128, 128),
        # a serving batch's step: each request's token joins its unfinished page
        append("append 128 x 1", 128, 1, 1000, 9000, 8, 128, 128),
        # prompt chunks of odd lengths: whole pages written, half of each key rotated
        append("append 4 x 4001", 4, 4001, 4033, 16401, 8, 128, 64),
        # one token of one request: the cache split over the GPU, latency
        read("attn", "attn one token, 4k", 1, 1, 32, 8, 128, 4096, 4096),
        # a serving batch of mixed lengths on shuffled pages: the cache's bytes
        read("attn", "attn 64 rows, 4k-64k", 64, 1, 64, 8, 128, 4096, 65536),
        # speculative verify: anchor and five drafts per request, seven heads to a key head, rotated queries
        read("attn", "attn verify 32 x 6", 32, 6, 28, 4, 64, 4099, 6143, turn=64),
        # chunked prefill: 512 new rows per request over their history: arithmetic
        read("attn", "attn extend 4 x 512", 4, 512, 32, 8, 128, 8320, 16512),
        # one long request: its pages ranked for one token
        read("select", "select one token, 128k", 1, 1, 32, 8, 128, 131072, 131072, turn=128, blocks=32),
        # every row of prompt chunks ranks its own pages
        read("select", "select extend 4 x 512", 4, 512, 32, 8, 128, 8320, 16512, blocks=16),
        # the same long request's token over the selected pages: latency
        read("blocks", "blocks one token, 128k", 1, 1, 32, 8, 128, 131072, 131072, turn=128, blocks=32),
        # a serving batch that reads 64 pages a row whatever its length
        read("blocks", "blocks 64 rows, 4k-64k", 64, 1, 64, 8, 128, 4096, 65536, blocks=64),
        # prompt chunks, each row over its own pages
        read("blocks", "blocks extend 4 x 512", 4, 512, 32, 8, 128, 8320, 16512, blocks=16),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    kind = rng.choice(["append", "attn", "select", "blocks"])
    kv_heads, dim, turn = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128]), rng.choice([0, 1, 2])
    turn = (0, dim // 2, dim)[turn]
    if kind == "append":
        new = log(1, 5000)
        requests = log(1, max(1, min(128, 100000 // (new * kv_heads))))
        lo = new + log(1, 9000)
        return {"kind": kind, "requests": requests, "new": new, "lo": lo, "hi": lo + rng.choice([0, 63, 2000]),
                "kv_heads": kv_heads, "dim": dim, "turn": turn}
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    rows = rng.choice([1, 1, log(2, 9), log(10, 512)])
    # bounded by the largest listed cases: tokens of the padded caches, attended pairs, listed pages' bytes
    requests = log(1, max(1, min(64, 60000 // (rows * heads))))
    blocks = log(4, 64)
    hi = int(min(131072, 2e9 / (requests * kv_heads * dim), 1e9 / (requests * rows * heads) * 128 / dim))
    if kind == "blocks":
        blocks = max(4, min(blocks, int(6e9 / (requests * rows * kv_heads * BLOCK * dim * 4))))
    b = max(rows, log(rows + 32, max(hi, rows + 33)))
    lo = max(rows, b // rng.choice([1, 2, 3]))
    if kind == "select":  # more pages than are selected
        lo = max(lo, rows + (blocks + 2) * BLOCK)
    return {"kind": kind, "requests": requests, "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "lo": lo, "hi": max(b, lo), "turn": turn,
            "blocks": blocks if kind in ("select", "blocks") else 0}


def lengths(n, lo, hi):
    """n context lengths spread evenly over the logarithm of [lo, hi], in a fixed mixed order."""
    span = [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]
    step = next(s for s in (7, 11, 13, 5, 3, 1) if math.gcd(s, n) == 1)
    return [span[i * step % n] for i in range(n)]


def counts(case):
    """New tokens of each request of an append: ragged where there are many."""
    return [max(1, case["new"] - (i * 37) % max(1, case["new"] // 8)) for i in range(case["requests"])]


# ---- inputs -------------------------------------------------------------------------
def fill_pages(pool, heads, dim, gen):
    """Every page: N(0, 1) keys and values, one channel in 16 of each head four times as large (as trained
    keys have them), quantised by page and head."""
    side = BLOCK * dim
    wide = 1 + 3 * (torch.rand(2, heads, dim, generator=gen, device=pool.device) < 1 / 16)
    for p in range(0, pool.shape[0], 512):
        n = min(512, pool.shape[0] - p)
        for k in range(2):
            x = torch.randn(n, heads, BLOCK, dim, generator=gen, device=pool.device) * wide[k][:, None]
            s = x.abs().amax((-1, -2)) / 448
            code = (x / s[..., None, None]).to(E4M3).view(torch.uint8)
            pool[p:p + n, :, k * side:(k + 1) * side] = (keys_in, values_in)[k](code)
            pool[p:p + n, :, 2 * side + 4 * k:2 * side + 4 * k + 4] = s.view(torch.uint8).view(n, heads, 4)
    pool[..., 2 * side + 8:] = 0


def keys_in(x):
    """[..., 64 tokens, dim] codes to a page's order of keys: 16-byte pieces of 8 tokens together."""
    d = x.shape[-1]
    return x.unflatten(-1, (d // 16, 16)).unflatten(-3, (8, 8)).transpose(-3, -2).flatten(-4)


def values_in(x):
    """[..., 64 tokens, dim] codes to a page's order of values: transposed, 16 tokens of 8 dims together."""
    d = x.shape[-1]
    x = x.transpose(-1, -2).unflatten(-1, (4, 16)).unflatten(-3, (d // 8, 8))
    return x.transpose(-3, -2).flatten(-4)


def keys_out(x, d):
    return x.unflatten(-1, (8, d // 16, 8, 16)).transpose(-3, -2).flatten(-4, -3).flatten(-2)


def values_out(x, d):
    return x.unflatten(-1, (d // 8, 4, 8, 16)).transpose(-3, -2).flatten(-4, -3).flatten(-2).transpose(-1, -2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (prepare_append if case["kind"] == "append" else prepare_read)(case, gen, "cuda")


def tables(rows, turn, gen, dev):
    if not turn:
        return None, None
    th = torch.rand(rows, turn // 2, generator=gen, device=dev) * (2 * math.pi)
    return torch.cos(th), torch.sin(th)


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare_append(case, gen, dev):
    B, H, d = case["requests"], case["kv_heads"], case["dim"]
    new = counts(case)
    end = [max(e, k) for e, k in zip(lengths(B, case["lo"], case["hi"]), new)]
    pos0 = [e - k for e, k in zip(end, new)]
    width = -(-max(end) // BLOCK)
    held = [range(p // BLOCK, (e - 1) // BLOCK + 1) for p, e in zip(pos0, end)]
    units = sum(len(h) for h in held)
    n = units + 3
    ids = torch.randperm(n, generator=gen, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, h in enumerate(held):
        table[b, h.start:h.stop] = ids[at:at + len(h)]
        at += len(h)
    off = [0]
    for k in new:
        off.append(off[-1] + k)
    pool = torch.zeros(n, H, 2 * BLOCK * d + 128, dtype=torch.uint8, device=dev)
    tail = torch.randn(B, H, 2, RING, d, generator=gen, device=dev).bfloat16()
    s = {"case": case, "pool": pool, "table": table, "tail": tail, "tail0": tail.clone(), "units": units,
         "codes": torch.zeros(n, H, d, dtype=torch.int8, device=dev), "ss": torch.zeros(n, H, device=dev),
         "pos0": ints(pos0, dev), "off": ints(off, dev), "tokens": off[-1],
         "k": torch.randn(off[-1], H, d, generator=gen, device=dev).bfloat16(),
         "v": torch.randn(off[-1], H, d, generator=gen, device=dev).bfloat16()}
    s["cos"], s["sin"] = tables(max(end), case["turn"], gen, dev)
    if own:  # what a serving program sets up once for its cache
        import fp4_sparse_attention_csa_gb300 as csa
        s["cache"] = csa.make_kv8(pool, tail, table, n, H, d, s["codes"], s["ss"])
        s["rope"] = csa.make_rope(s["cos"], s["sin"]) if case["turn"] else None
        s["ws"] = torch.zeros(csa.csa_workspace_size(csa.OP_KV8_APPEND, 0, 0, 0), dtype=torch.uint8, device=dev)
    return s


def prepare_read(case, gen, dev):
    B, r, H, KH, d = case["requests"], case["rows"], case["heads"], case["kv_heads"], case["dim"]
    ctx = torch.tensor(lengths(B, case["lo"], case["hi"])).clamp_min(r)
    pages = [-(-int(c) // BLOCK) for c in ctx]
    n, width = sum(pages), max(pages)
    pool = torch.empty(n, KH, 2 * BLOCK * d + 128, dtype=torch.uint8, device=dev)
    if case["kind"] != "select":
        fill_pages(pool, KH, d, gen)
    ids = torch.randperm(n, generator=gen, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = ids[at:at + k]
        at += k
    R, M = B * r, case["blocks"]
    s = {"case": case, "pool": pool, "table": table, "most": int(ctx.max()),
         "tail": torch.zeros(B, KH, 2, RING, d, dtype=torch.bfloat16, device=dev),
         "req": torch.arange(B, device=dev).repeat_interleave(r).int(),
         "pos": (ctx[:, None] - r + torch.arange(r)).reshape(-1).int().to(dev),
         "q": torch.randn(R, H, d, generator=gen, device=dev).bfloat16(), "scale": 1 / math.sqrt(d),
         "codes": None, "ss": None}
    s["cos"], s["sin"] = tables(s["most"], case["turn"], gen, dev)
    if case["kind"] == "select":
        mean = torch.randn(n, KH, d, generator=gen, device=dev) / 8
        mean += 0.3 * torch.randn(KH, d, generator=gen, device=dev)  # what a head's keys have in common
        s["ss"] = mean.abs().amax(-1) / 127
        s["codes"] = (mean / s["ss"][..., None]).round().to(torch.int8)
        s["out"] = torch.empty(R, KH, M, dtype=torch.int32, device=dev)
    else:
        s["out"] = torch.empty(R, H, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(R, H, dtype=torch.float32, device=dev)
    if case["kind"] == "blocks":  # the first page, the row's last two, and the rest spread over its context
        j = torch.arange(width, device=dev)
        last = (s["pos"] // BLOCK)[:, None, None]
        key = torch.rand(R, KH, width, generator=gen, device=dev)
        key = torch.where((j == 0) | (j > last - 2), 2.0, key).masked_fill(j > last, -1.0)
        top = torch.topk(key, min(M, width), -1)
        lists = torch.where(top.values >= 0, top.indices, width).sort(-1).values
        lists = torch.where(lists < width, lists, -1).int()
        s["lists"] = torch.nn.functional.pad(lists, (0, M - lists.shape[-1]), value=-1).contiguous()
    if own:  # what a serving program sets up once for its cache and its step
        import fp4_sparse_attention_csa_gb300 as csa
        s["cache"] = csa.make_kv8(pool, s["tail"], table, n, KH, d, s["codes"], s["ss"])
        s["rope"] = csa.make_rope(s["cos"], s["sin"]) if case["turn"] else None
        s["rows"] = csa.make_rows(s["req"], s["pos"], s["most"], r)
        op, h = (csa.OP_KV8_SELECT, KH) if case["kind"] == "select" else (csa.OP_KV8_ATTN, H)
        s["ws"] = torch.zeros(csa.csa_workspace_size(op, R, s["most"], h), dtype=torch.uint8, device=dev)
    return s


# ---- one pass -----------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["kind"] == "append":
        if case["new"] > BLOCK:  # such a call overwrites what it reads of the ring: each pass starts from the same one
            s["tail"].copy_(s["tail0"])
        if own:
            import fp4_sparse_attention_csa_gb300 as csa
            csa.csa_kv8_append(s["cache"], s["rope"], s["pos0"], s["off"], s["tokens"], s["k"], s["v"], s["ws"])
        else:
            plain_append(s)
        side = 2 * BLOCK * case["dim"]
        return s["pool"][..., :side].view(E4M3), s["pool"][..., side:].view(torch.float32), s["tail"], s["codes"], s["ss"]
    if case["kind"] == "select":
        if own:
            import fp4_sparse_attention_csa_gb300 as csa
            csa.csa_kv8_select(s["cache"], s["rows"], case["heads"], s["q"], s["rope"], case["blocks"], 1, 2, s["out"],
                               s["ws"])
            return s["out"]
        return plain_select(s)
    if own:
        import fp4_sparse_attention_csa_gb300 as csa
        if case["kind"] == "attn":
            csa.csa_kv8_attn(s["cache"], s["rows"], case["heads"], s["q"], s["rope"], s["scale"], s["out"], s["lse"],
                             s["ws"])
        else:
            csa.csa_kv8_block_attn(s["cache"], s["rows"], s["lists"], case["blocks"], case["heads"], s["q"], s["rope"],
                                   s["scale"], s["out"], s["lse"], s["ws"])
        return s["out"], s["lse"]
    return plain_attn(s) if case["kind"] == "attn" else plain_blocks(s)


def turned(x, s, pos):
    """x [..., heads, dim] in bf16, its first `turn` dims rotated by halves at pos [...]: as a model holds
    rotated queries and keys, in bf16."""
    x, n = x.float(), s["case"]["turn"]
    if not n:
        return x
    c, t = s["cos"][pos][..., None, :], s["sin"][pos][..., None, :]
    a, b = x[..., :n // 2], x[..., n // 2:n]
    return torch.cat([a * c - b * t, b * c + a * t, x[..., n:]], -1).bfloat16().float()


def divided(a, b):
    """a / b rounded once (a number in its place would be turned into its reciprocal first)."""
    return torch.full_like(b, a) / b if isinstance(a, (int, float)) else a / torch.full_like(a, b)


def plain_append(s):
    B, d = s["case"]["requests"], s["case"]["dim"]
    dev = s["k"].device
    pos0, off = s["pos0"].long(), s["off"].long()
    n = off[1:] - off[:-1]
    tok = torch.arange(s["tokens"], device=dev)
    of = torch.repeat_interleave(torch.arange(B, device=dev), n, output_size=s["tokens"])
    new = torch.stack([turned(s["k"], s, pos0[of] + tok - off[of]), s["v"].float()], 2)      # [tokens, heads, 2, dim]
    # the pages that the call touches, and each one's tokens
    j0 = pos0 // BLOCK
    each = torch.where(n > 0, (pos0 + n - 1) // BLOCK - j0 + 1, 0)
    b = torch.repeat_interleave(torch.arange(B, device=dev), each, output_size=s["units"])
    j = j0[b] + torch.arange(s["units"], device=dev) - (each.cumsum(0) - each)[b]
    pos = (j * BLOCK)[:, None] + torch.arange(BLOCK, device=dev)
    is_new = (pos >= pos0[b][:, None]) & (pos < (pos0 + n)[b][:, None])
    is_old = pos < pos0[b][:, None]
    x = new[(off[b] - pos0[b])[:, None].add(pos).clamp(0, s["tokens"] - 1)].movedim(1, 3)   # [units, heads, 2, 64, dim]
    old = s["tail"][b[:, None], :, :, pos % RING].float().movedim(1, 3)
    x = torch.where(is_new[:, None, None, :, None], x, torch.where(is_old[:, None, None, :, None], old, 0.0))
    # a token that is not all numbers: its key is NaN, and it counts for nothing else
    bad = ~torch.isfinite(x).all(-1).all(2)[:, :, None, :, None]
    x = torch.where(bad, 0.0, x)
    top = x.abs().amax((-1, -2))
    inv = torch.where(top >= 2.0 ** -100, divided(448.0, top), 0.0)
    scale = torch.where(top >= 2.0 ** -100, divided(top, 448.0), 0.0)
    code = (x * inv[..., None, None]).clamp(-448, 448)
    key = torch.where(bad[:, :, 0], math.nan, code[:, :, 0]).to(E4M3).view(torch.uint8)
    page = s["table"][b, j].long()
    side = BLOCK * d
    s["pool"][page, :, :side] = keys_in(key)
    s["pool"][page, :, side:2 * side] = values_in(code[:, :, 1].to(E4M3).view(torch.uint8))
    s["pool"][page, :, 2 * side:2 * side + 8] = scale.contiguous().view(torch.uint8)
    # summary: the mean of the page's keys, in a fixed order of sums
    q = x[:, :, 0].unflatten(2, (4, 16))
    part = q[..., 0, :] + q[..., 1, :]
    for i in range(2, 16):
        part = part + q[..., i, :]
    mean = ((part[:, :, 0] + part[:, :, 1]) + (part[:, :, 2] + part[:, :, 3])) * (1 / BLOCK)
    top = mean.abs().amax(-1)
    inv = torch.where(top >= 2.0 ** -100, divided(127.0, top), 0.0)
    s["codes"][page] = (mean * inv[..., None]).round().clamp(-127, 127).to(torch.int8)
    s["ss"][page] = torch.where(top >= 2.0 ** -100, divided(top, 127.0), 0.0)
    # the ring holds each request's last 128 tokens
    last = (pos0 + n - 1)[:, None]
    at = last - (last - torch.arange(RING, device=dev)) % RING
    take = (at >= pos0[:, None]) & (n > 0)[:, None]
    ring = new[(off[:-1] - pos0)[:, None].add(at).clamp(0, s["tokens"] - 1)].movedim(1, 3)
    s["tail"].copy_(torch.where(take[:, None, None, :, None], ring, s["tail"].float()))


def dequantised(s, pages):
    """Keys and values [..., heads, 64, dim] of pages."""
    d = s["case"]["dim"]
    side = BLOCK * d
    raw = s["pool"][pages]
    scale = raw[..., 2 * side:2 * side + 8].contiguous().view(torch.float32)
    key = keys_out(raw[..., :side], d).contiguous().view(E4M3).float() * scale[..., 0, None, None]
    return key, values_out(raw[..., side:2 * side], d).contiguous().view(E4M3).float() * scale[..., 1, None, None]


def softmax_over(logit, value):
    """logit [..., rows, keys], value [..., keys, dim]: (out, lse); a row of no key gives 0 and -inf."""
    m = logit.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(logit - m)
    l = p.sum(-1, keepdim=True)
    o = p @ value
    return torch.where(l > 0, o / l, 0.0), torch.where(l > 0, m + torch.log(l), LOWEST)[..., 0]


def plain_attn(s):
    case = s["case"]
    B, r, H, KH, d = case["requests"], case["rows"], case["heads"], case["kv_heads"], case["dim"]
    key, value = (x.transpose(1, 2).flatten(2, 3) for x in dequantised(s, s["table"].long().clamp_min(0)))  # [B, KH, n, d]
    q = turned(s["q"], s, s["pos"].long()).view(B, r, KH, H // KH, d).transpose(1, 2).flatten(2, 3)
    logit = (q @ key.transpose(-1, -2)) * s["scale"]
    hidden = torch.arange(key.shape[2], device=q.device) > s["pos"].view(B, r, 1)
    logit.view(B, KH, r, H // KH, -1).masked_fill_(hidden[:, None, :, None], LOWEST)
    o, lse = softmax_over(logit, value)
    o = o.view(B, KH, r, H // KH, d).transpose(1, 2).reshape(B * r, H, d)
    return o.bfloat16(), lse.view(B, KH, r, H // KH).transpose(1, 2).reshape(B * r, H)


def plain_blocks(s):
    case = s["case"]
    R, H, KH, d = s["q"].shape[0], case["heads"], case["kv_heads"], case["dim"]
    lists = s["lists"].long()                                                            # [R, KH, M]
    page = s["table"][s["req"].long()[:, None, None], lists.clamp_min(0)].long()
    head = torch.arange(KH, device=page.device)[:, None]
    side = BLOCK * d
    raw = s["pool"][page, head]                                                          # [R, KH, M, bytes]
    scale = raw[..., 2 * side:2 * side + 8].contiguous().view(torch.float32)
    key = (keys_out(raw[..., :side], d).contiguous().view(E4M3).float() * scale[..., 0, None, None]).flatten(2, 3)
    value = values_out(raw[..., side:2 * side], d).contiguous().view(E4M3).float() * scale[..., 1, None, None]
    at = lists[..., None] * BLOCK + torch.arange(BLOCK, device=page.device)
    seen = (lists[..., None] >= 0) & (at <= s["pos"][:, None, None, None])
    q = turned(s["q"], s, s["pos"].long()).view(R, KH, H // KH, d)
    logit = (q @ key.transpose(-1, -2)) * s["scale"]
    logit = logit.masked_fill(~seen.flatten(2)[:, :, None], LOWEST)
    o, lse = softmax_over(logit, value.flatten(2, 3))
    return o.reshape(R, H, d).bfloat16(), lse.reshape(R, H)


def plain_select(s):
    case = s["case"]
    B, r, H, KH, d, M = case["requests"], case["rows"], case["heads"], case["kv_heads"], case["dim"], case["blocks"]
    pos = s["pos"].long()
    q = turned(s["q"], s, pos)
    top = q.abs().amax(-1)
    inv = torch.where(top >= 2.0 ** -100, divided(127.0, top), 0.0)
    sq = torch.where(top >= 2.0 ** -100, divided(top, 127.0), 0.0)
    code = (q * inv[..., None]).round().clamp(-127, 127).view(B, r, KH, H // KH, d)
    pages = s["table"].long().clamp_min(0)
    key = s["codes"][pages].float().transpose(1, 2)                                      # [B, KH, width, d]
    dot = code.transpose(1, 2).flatten(2, 3) @ key.transpose(-1, -2)                     # whole numbers below 2^24
    dot = dot.view(B, KH, r, H // KH, -1) * sq.view(B, r, KH, H // KH).transpose(1, 2)[..., None]
    score = dot.amax(3) * s["ss"][pages].transpose(1, 2)[:, :, None]                     # [B, KH, r, width]
    j = torch.arange(pages.shape[1], device=q.device)
    last = (pos // BLOCK).view(B, 1, r, 1)
    score = torch.where((j < 1) | (j > last - 2), math.inf, score).masked_fill(j > last, LOWEST)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :M]      # ties to the lowest page
    width = pages.shape[1]
    best = torch.where(best <= last, best, width).sort(-1).values
    best = torch.where(best < width, best, -1).transpose(1, 2).reshape(B * r, KH, -1).int()
    return torch.nn.functional.pad(best, (0, M - best.shape[-1]), value=-1)


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    KH, d = case["kv_heads"], case["dim"]
    record = KH * (2 * BLOCK * d + 8)
    if case["kind"] == "append":
        new = counts(case)
        end = [max(e, k) for e, k in zip(lengths(case["requests"], case["lo"], case["hi"]), new)]
        token = KH * 2 * d * 2
        touched = sum((e - 1) // BLOCK - (e - k) // BLOCK + 1 for e, k in zip(end, new))
        earlier = sum((e - k) % BLOCK for e, k in zip(end, new))
        return {"bytes": (sum(new) + earlier + sum(min(k, RING) for k in new)) * token + touched * (record + KH * (d + 4))
                + sum(new) * case["turn"] * 4, "flops": 0}
    B, r, H, M = case["requests"], case["rows"], case["heads"], case["blocks"]
    ctx = [max(c, r) for c in lengths(B, case["lo"], case["hi"])]
    q = B * r * H * d * 2
    if case["kind"] == "select":
        pages = [-(-c // BLOCK) for c in ctx]
        return {"bytes": sum(pages) * KH * (d + 4) + q + B * r * KH * M * 4, "flops": sum(pages) * r * H * d * 2}
    if case["kind"] == "attn":
        return {"bytes": sum(-(-c // BLOCK) for c in ctx) * record + q * 2 + B * r * H * 4,
                "flops": sum(p + 1 for c in ctx for p in range(c - r, c)) * H * d * 4}
    pages = [min(M, -(-c // BLOCK)) for c in ctx]
    return {"bytes": sum(min(k * r, -(-c // BLOCK)) for k, c in zip(pages, ctx)) * record + q * 2 + B * r * (H + KH * M) * 4,
            "flops": sum(pages) * r * BLOCK * H * d * 4}


# ---- the definition in 64 bits ------------------------------------------------------
def e4m3(byte):
    byte = byte.long()
    e, m = (byte >> 3) & 15, (byte & 7).to(F64)
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).to(F64)), m * 2.0 ** -9)
    return torch.where(byte > 127, -v, v)


def rotation(s, x, pos):
    """Dims i and i + turn / 2 as a complex number, turned; each product and sum is rounded to 32 bits and the
    result to bf16, as the definition has it."""
    n = s["case"]["turn"]
    y = x.float().clone()
    for i in range(n // 2):
        c, t = s["cos"][pos, i][:, None], s["sin"][pos, i][:, None]
        re, im = x[..., i].float(), x[..., i + n // 2].float()
        y[..., i], y[..., i + n // 2] = re.mul(c).sub(im.mul(t)), im.mul(c).add(re.mul(t))
    return y.bfloat16().to(F64)


def exact_append(case, s):
    B, KH, d = case["requests"], case["kv_heads"], case["dim"]
    side = BLOCK * d
    pool = s["pool"].to(F64)
    code = e4m3(s["pool"][..., :2 * side])
    scale, tail, ss = pool[..., :32].clone().zero_(), s["tail"].to(F64), s["ss"].to(F64)
    off, pos0 = s["off"].tolist(), s["pos0"].tolist()
    t = torch.arange(BLOCK, device="cuda")
    for b in range(B):
        lo, hi = pos0[b], pos0[b] + off[b + 1] - off[b]
        at = torch.arange(lo, hi, device="cuda")
        both = torch.stack([rotation(s, s["k"][off[b]:off[b + 1]], at), s["v"][off[b]:off[b + 1]].to(F64)])
        for j in range(lo // BLOCK, (hi - 1) // BLOCK + 1):
            first = j * BLOCK
            x = torch.zeros(2, BLOCK, KH, d, dtype=F64, device="cuda")
            for k in range(2):
                if first < lo:
                    ring = torch.arange(first, lo, device="cuda") % RING
                    x[k, :lo - first] = s["tail"][b, :, k, ring].to(F64).transpose(0, 1)
                a, z = max(first, lo), min(first + BLOCK, hi)
                x[k, a - first:z - first] = both[k, a - lo:z - lo]
            page = int(s["table"][b, j])
            top = x.abs().amax((1, 3))                                                   # [2, KH]
            y = x / (top / 448)[:, None, :, None]
            for tok in range(0, BLOCK, 8):  # eight tokens of a 16-byte piece of dims, pieces one after another
                part = y[0, tok:tok + 8].permute(1, 2, 0).reshape(KH, d // 16, 16, 8).permute(0, 1, 3, 2)
                code[page, :, tok * d:(tok + 8) * d] = part.reshape(KH, -1)
            where = (torch.arange(d, device="cuda")[:, None] // 8 * 512 + t // 16 * 128
                     + torch.arange(d, device="cuda")[:, None] % 8 * 16 + t % 16)
            code[page, :, side + where] = y[1].permute(1, 2, 0)
            scale[page, :, 0], scale[page, :, 1] = top[0] / 448, top[1] / 448
            ss[page] = x[0].mean(0).abs().amax(-1) / 127
        keep = max(lo, hi - RING)
        tail[b, :, :, torch.arange(keep, hi, device="cuda") % RING] = both[:, keep - lo:].permute(2, 0, 1, 3)
    return code, scale, tail, None, ss


def exact(case, seed):
    """Request by request and head by head, a code's value from its sign, exponent and fraction bits."""
    if case["kind"] == "select":
        return None
    s = prepare(case, seed)
    if case["kind"] == "append":
        return exact_append(case, s)
    B, r, H, KH, d = case["requests"], case["rows"], case["heads"], case["kv_heads"], case["dim"]
    G, side = H // KH, BLOCK * d
    t, dim = torch.arange(BLOCK, device="cuda"), torch.arange(d, device="cuda")
    kat = t[:, None] // 8 * 8 * d + dim // 16 * 128 + t[:, None] % 8 * 16 + dim % 16
    vat = side + dim // 8 * 512 + t[:, None] // 16 * 128 + dim % 8 * 16 + t[:, None] % 16
    out = torch.zeros(B * r, H, d, dtype=F64, device="cuda")
    lse = torch.full((B * r, H), LOWEST, dtype=F64, device="cuda")
    for b in range(B):
        pos = s["pos"][b * r:(b + 1) * r].long()
        n = int(pos[-1]) // BLOCK + 1
        rows = rotation(s, s["q"][b * r:(b + 1) * r], pos).view(r, KH, G, d)
        for h in range(KH):
            raw = s["pool"][s["table"][b, :n].long(), h]
            sc = raw[:, 2 * side:2 * side + 8].contiguous().view(torch.float32).to(F64)
            key = (e4m3(raw[:, kat]) * sc[:, 0, None, None]).view(-1, d)
            value = (e4m3(raw[:, vat]) * sc[:, 1, None, None]).view(-1, d)
            for lo in range(0, r, 128):
                p, q = pos[lo:lo + 128], rows[lo:lo + 128, h]
                see = torch.arange(n * BLOCK, device="cuda") <= p[:, None]
                if case["kind"] == "blocks":
                    member = torch.zeros(len(p), n + 1, dtype=torch.bool, device="cuda")
                    chosen = s["lists"][b * r + lo:b * r + lo + len(p), h].long()
                    member.scatter_(1, torch.where(chosen >= 0, chosen, n), True)
                    see &= member[:, :n].repeat_interleave(BLOCK, 1)
                w = (q.reshape(-1, d) @ key.T).view(len(p), G, -1) * s["scale"]
                w = w.masked_fill(~see[:, None], LOWEST)
                z = torch.logsumexp(w, -1)
                o = (torch.exp(w - z[..., None]).view(-1, n * BLOCK) @ value).view(len(p), G, d)
                at = slice(b * r + lo, b * r + lo + len(p))
                out[at, h * G:(h + 1) * G], lse[at, h * G:(h + 1) * G] = o, z
    return out, lse
