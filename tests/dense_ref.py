"""Dense attention over the paged FP4 cache in 64 bits, from the byte layout,
and the error that the kernel's roundings allow."""
import numpy as np
import torch

D, WIN, PAGE = 512, 128, 64
_E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b):
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(1 + m / 8.0, e - 7), m * 2.0 ** -9)
    return np.where(b > 127, -v, v)


def entries(kv_pool, table_row, n, num_pages):
    """(values [n, 512], whether each entry's page is in the pool)."""
    pool = np.asarray(kv_pool).reshape(-1, 18432)
    pg = np.asarray(table_row)[np.arange(n) // PAGE]
    ok = (pg >= 0) & (pg < num_pages)
    pg, slot = np.where(ok, pg, 0), np.arange(n) % PAGE
    data = pool[pg[:, None], (256 * slot)[:, None] + np.arange(256)]
    sc = e4m3(pool[pg[:, None], (16384 + 32 * slot)[:, None] + np.arange(32)])
    v = np.stack([_E2M1[data & 15], _E2M1[data >> 4]], -1).reshape(n, 32, 16) * sc[:, :, None]
    return v.reshape(n, D), ok


def rotate(x, cos, sin):
    a, b = x[..., 448:480].copy(), x[..., 480:].copy()
    y = x.copy()
    y[..., 448:480], y[..., 480:] = a * cos - b * sin, b * cos + a * sin
    return y


def row_reference(kv_pool, table_row, num_pages, P, pos, q, scale, win=None, rope=None):
    """(out [H, 512], lse [H], bound on out, bound on lse) of one row in float64.
    win: (codes [cap, 512], scales [cap]) of its request; rope: (cos, sin)."""
    n = (pos + 1) // P
    keys, ok = entries(kv_pool, table_row, n, num_pages)
    keys = keys[ok]
    q = np.asarray(q, np.float64)
    rot = np.zeros((len(keys), 1))
    if rope is not None:
        q = rotate(q, rope[0][pos].astype(np.float64), rope[1][pos].astype(np.float64))
    if win is not None:
        p = np.arange(max(0, pos - WIN + 1), pos + 1)
        cap = win[1].shape[0]
        w = e4m3(win[0][p % cap]) * win[1][p % cap].astype(np.float64)[:, None]
        if rope is not None:
            w = rotate(w, rope[0][p].astype(np.float64), rope[1][p].astype(np.float64))
        keys = np.concatenate([keys, w])
        rot = np.concatenate([rot, np.ones((len(w), 1))])
    H = q.shape[0]
    if len(keys) == 0:
        z = np.zeros((H, D))
        return z, np.full(H, -np.inf), z, np.zeros(H)
    logit = (q @ keys.T) * scale
    m = logit.max(-1, keepdims=True)
    p = np.exp(logit - m)
    l = p.sum(-1, keepdims=True)
    out = p @ keys / l
    # Logits: 32 accumulations of 16 exact products, each off by at most one step
    # (2^-22) of the sum of magnitudes; the factor, the max and exp2 in fp32.
    # Rotated query values carry 22 bits, rotated window values 11 (fp16).
    mag = (np.abs(q) @ np.abs(keys).T) * abs(scale)
    delta = 2.0 ** -17 * mag + 2.0 ** -21 * (4 + np.abs(logit) + np.abs(m))
    if rope is not None:
        rotmag = (np.abs(q[:, 448:]) @ np.abs(keys[:, 448:]).T) * abs(scale)
        delta = delta + rotmag * (2.0 ** -22 + 2.0 ** -11 * rot.T)
    wt = p / l
    # P rounded to fp16: 2^-11, or half its smallest step (2^-25) where p is below
    # 2^-14, relative to a running max that may lie 2^14 below the row's; then
    # len/16 accumulations, the sums of p and the parts' merge.
    step = 2.0 ** -11 + (len(keys) / 16 + 96) * 2.0 ** -22
    A = np.abs(keys)
    bound = (wt * (2 * delta + step)) @ A + (delta * wt).sum(-1, keepdims=True) * np.abs(out)
    bound += 2.0 ** -25 * A.sum(0) / l
    if rope is not None:
        Ar = np.abs(keys * rot)
        Ar[:, :448] = 0
        bound += 2.0 ** -11 * wt @ Ar
    bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out) + 1e-38
    lse = (m + np.log(l))[:, 0]
    lse_bound = (delta * wt).sum(-1) * 2 + 2.0 ** -20 * (4 + np.abs(lse))
    return out, lse, bound, lse_bound


class Case:
    """A cache of random entries (any bytes but NaN scales), a window and rows."""

    def __init__(self, seed, ctx, P, win_cap=0, spread=1.0, extra_pages=3, device="cuda"):
        g = np.random.default_rng(seed)
        self.P, self.device, self.B = P, device, len(ctx)
        held = [max(1, -(-(c // P) // PAGE)) for c in ctx]
        self.num_pages = sum(held) + extra_pages
        self.kv = g.integers(0, 256, (self.num_pages, 18432), dtype=np.uint8)
        lo, hi = int(56 - 12 * spread), int(56 + 4 * spread)          # E4M3 scales around 1, some zero
        sc = g.integers(lo, hi, (self.num_pages, 2048), dtype=np.uint8)
        sc[g.random(sc.shape) < 0.02] = 0
        self.kv[:, 16384:] = sc
        self.table = np.full((self.B, max(held) + 1), -1, np.int32)
        ids, at = g.permutation(self.num_pages).astype(np.int32), 0
        for b, k in enumerate(held):
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.cap = win_cap
        if win_cap:
            codes = g.integers(0, 256, (self.B, win_cap, D), dtype=np.uint8)
            codes[(codes & 127) == 127] = 0
            self.codes = codes
            self.wscale = (0.01 * np.exp2(g.uniform(-2, 2, (self.B, win_cap)))).astype(np.float32)
            self.wscale[g.random(self.wscale.shape) < 0.03] = 0
        self.g = g

    def queries(self, R, H, scale=1.0):
        q = torch.from_numpy((self.g.standard_normal((R, H, D)) * scale).astype(np.float32)).bfloat16()
        return q

    def run(self, csa, req, pos, H, q, scale=512 ** -0.5, rope=None, lse=True, mrpr=None, max_entries=None):
        dev = self.device
        self.d_kv = torch.from_numpy(self.kv).to(dev)
        self.d_idx = torch.zeros(self.num_pages, 4352, dtype=torch.uint8, device=dev)
        self.d_table = torch.from_numpy(self.table).to(dev)
        self.cache = csa.make_cache(self.d_kv, self.d_idx, self.d_table, self.num_pages, self.P)
        self.window = None
        if self.cap:
            self.d_codes, self.d_wscale = torch.from_numpy(self.codes).to(dev), torch.from_numpy(self.wscale).to(dev)
            self.window = csa.make_window(self.d_codes, self.d_wscale, self.cap)
        R = len(req)
        self.d_req = torch.tensor(req, dtype=torch.int32, device=dev)
        self.d_pos = torch.tensor(pos, dtype=torch.int32, device=dev)
        ent = max([(p + 1) // self.P for p in pos] + [0]) if max_entries is None else max_entries
        per = max([list(req).count(b) for b in set(req)] + [1]) if mrpr is None else mrpr
        self.rows = csa.make_rows(self.d_req, self.d_pos, ent, per)
        self.d_q = q.to(dev)
        self.out = torch.full((R + 2, H, D), 7.0, dtype=torch.bfloat16, device=dev)
        self.lse = torch.full((R + 2, H), 7.0, device=dev) if lse else None
        self.opts = None
        if rope is not None:
            self.d_rope = [torch.from_numpy(t).to(dev) for t in rope]
            self.opts = csa.make_opts(rope_cos=self.d_rope[0], rope_sin=self.d_rope[1])
        # what a workspace held before must not matter past its status word
        self.ws = torch.full((csa.csa_workspace_size(csa.OP_DENSE_ATTN, R, ent, H),), 255, dtype=torch.uint8, device=dev)
        self.ws[:256] = 0
        self.call = lambda stream=None: csa.csa_dense_attn(self.cache, self.window, self.rows, H, self.d_q, scale,
                                                           self.out, self.lse, self.opts, self.ws, stream)
        self.call()
        return csa.csa_check_device_status(self.ws)

    def check(self, req, pos, H, q, scale=512 ** -0.5, rope=None, rows=None):
        R = len(req)
        out = self.out.double().cpu().numpy()
        lse = self.lse.double().cpu().numpy() if self.lse is not None else None
        qn = q.double().numpy()
        for r in (range(R) if rows is None else rows):
            b = req[r]
            win = (self.codes[b], self.wscale[b]) if self.cap else None
            o, z, tol, ztol = row_reference(self.kv, self.table[b], self.num_pages, self.P, pos[r], qn[r], scale, win, rope)
            err = np.abs(out[r] - o)
            assert (err <= tol).all(), (r, b, pos[r], float((err - tol).max()), float((err / np.maximum(tol, 1e-300)).max()))
            if lse is not None:
                fin = np.isfinite(z)
                assert np.array_equal(fin, np.isfinite(lse[r])) and (lse[r][~fin] == z[~fin]).all(), (r, lse[r], z)
                zerr = np.abs(lse[r][fin] - z[fin])
                assert (zerr <= ztol[fin]).all(), (r, float((zerr / ztol[fin]).max()))
        assert (out[R:] == 7.0).all()
        if lse is not None:
            assert (lse[R:] == 7.0).all()
