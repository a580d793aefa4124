"""Plain 64-bit statements of the paged-cache calls (include/fx.h), for tests: loops over sequences and heads,
numpy on the host.  Nothing here comes from the library."""
import numpy as np
import torch

D = 128
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table():
    """Value of every e4m3 byte: 4 exponent bits with bias 7, 3 mantissa bits; 0x7f and 0xff are NaN."""
    t = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        t[b] = -v if b & 128 else v
    return t


E4M3 = e4m3_table()


def nearest(x, grid):
    """Index of the entry of an ascending grid nearest to each x >= 0; a tie takes the even index."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x, exp=0):
    """(codes uint8 [..., 64], scale bytes uint8 [..., 8]) of fp64 rows [..., 128] whose values are bf16 values."""
    with np.errstate(invalid="ignore", over="ignore"):
        y = (np.asarray(x, np.float64) * 2.0 ** -exp).reshape(x.shape[:-1] + (8, 16))
        bad = ~np.isfinite(y).all(-1)
        y = np.where(bad[..., None], 0.0, y)
        a = np.abs(y).max(-1) / 6
        sb = np.maximum(nearest(np.minimum(a, 448.0), E4M3[:127]), 1)
        code = nearest(np.minimum(np.abs(y) / E4M3[sb][..., None], 6.0), GRID) | (np.signbit(y) << 3)
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 0x7f, sb).astype(np.uint8)


def dequantize(codes, scales, exp=0):
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (8, 16))
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    return (v * E4M3[scales][..., None]).reshape(codes.shape[:-1] + (D,)) * 2.0 ** exp


def bf16(x):
    """Nearest bf16 value of fp32 values, as fp64."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def rotate(x, cs, interleaved):
    """Rows x [n, heads, 128] (bf16 values) rotated by fp32 cs [n, rot]: (the stated result -- products and sums
    rounded to fp32, then bf16 -- and the same without any rounding), both fp64."""
    rot = cs.shape[-1]
    half = rot // 2
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    res = []
    for kind in (np.float32, np.float64):
        y = x.astype(kind)
        c, s = (cs[:, None, a].astype(kind) for a in (slice(0, half), slice(half, rot)))
        a, b = y[..., one].copy(), y[..., two].copy()
        y[..., one], y[..., two] = a * c - b * s, b * c + a * s
        res.append(y)
    return bf16(res[0]), res[1]


class Cache:
    """A paged cache on the host: pools of fp64 rows [n_pages, Hkv, page, 128] (what the pages hold), page table and
    lengths.  layout: "head" [page, head, row] storage, "row" [page, row, head], "gap" rows with room between them."""

    def __init__(self, fmt, lens, Hkv, page, seed=0, max_pages=None, layout="head", exps=(0, 0), garbage=True,
                 channel=1.0):
        g = np.random.default_rng(seed)
        self.fmt, self.lens, self.Hkv, self.page, self.exps = fmt, list(lens), Hkv, page, exps
        self.B = len(lens)
        need = [-(-n // page) for n in lens]
        self.max_pages = max_pages or max(max(need), 1)
        self.n_pages = sum(need) + 2
        order = g.permutation(self.n_pages)
        # entries of pages that hold no row in use are anything
        self.table = np.where(g.random((self.B, self.max_pages)) < 0.5, -7, 1 << 30).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.n_pages, Hkv, page, D)
        x = [bf16(g.standard_normal(shape) * (channel * 2.0 ** e)) for e in exps]
        self.layout = layout
        if fmt == "bf16":
            self.pool = x
        else:
            self.packed = [quantize(v, e) for v, e in zip(x, exps)]
            self.pool = [dequantize(c, s, e) for (c, s), e in zip(self.packed, exps)]
        self.garbage = garbage

    def spot(self, b, t):
        return self.table[b, t // self.page], t % self.page

    def used(self):
        """Mask [n_pages, page] of the rows in use."""
        m = np.zeros((self.n_pages, self.page), bool)
        for b, n in enumerate(self.lens):
            t = np.arange(n)
            m[self.spot(b, t)] = True
        return m

    def rows(self, which, b, h, at):
        at = np.asarray(at, np.int64)
        return self.pool[which][self.table[b, at // self.page], h, at % self.page]

    def device(self, fx, dev="cuda"):
        """The library's view.  Rows not in use hold NaN (bf16) or NaN scales and all-ones codes (4-bit)."""
        def lay(t):
            if self.layout == "head":
                return t.contiguous().to(dev)
            if self.layout == "row":
                return t.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3)
            w = t.shape[3]
            big = torch.zeros(t.shape[:3] + (w + 16 * 16,), dtype=t.dtype, device=dev)
            big[..., :w] = t.to(dev)
            return big[..., :w]
        un = torch.from_numpy(~self.used())[:, None, :, None]
        kw = {}
        if self.fmt == "bf16":
            k, v = (torch.from_numpy(p).to(torch.bfloat16) for p in self.pool)
            if self.garbage:
                k, v = (torch.where(un, torch.tensor(float("nan"), dtype=torch.bfloat16), t) for t in (k, v))
            k, v = lay(k), lay(v)
        else:
            (kc, ks), (vc, vs) = ((torch.from_numpy(c), torch.from_numpy(s)) for c, s in self.packed)
            if self.garbage:
                kc, vc, ks, vs = (torch.where(un, torch.tensor(255, dtype=torch.uint8), t) for t in (kc, vc, ks, vs))
            k, v = lay(kc), lay(vc)
            kw = dict(k_scale=lay(ks), v_scale=lay(vs), k_exp=self.exps[0], v_exp=self.exps[1])
        return fx.PagedKV(k, v, torch.from_numpy(self.table).to(dev),
                          torch.tensor(self.lens, dtype=torch.int32, device=dev), **kw)

    def keys(self, b, h, idx=None, tail_lo=None):
        """Cache rows that attention of (b, h) runs over, in order, duplicates included."""
        n = self.lens[b]
        lo = 0 if tail_lo is None else max(0, int(tail_lo[b]))
        tail = np.arange(lo, n, dtype=np.int64)
        if idx is None:
            return tail
        lst = np.asarray(idx[b, h], np.int64)
        return np.concatenate((lst[(lst >= 0) & (lst < n)], tail))


def attend(c, q, scale, idx=None, tail_lo=None):
    """fx_paged_decode in 64 bits: (out [B, Hq, Mq, 128], lse [B, Hq, Mq], mag [B, Hq, Mq, 128], dl [B, Hq, Mq],
    far [B, Hq, Mq, 128]).  mag = sum p |v|; far = sum |v|; dl = the largest scale * sum_d |q_d k_d| of a row (what
    a logit's error is relative to)."""
    q = np.asarray(q, np.float64)
    B, Hq, Mq, _ = q.shape
    G = Hq // c.Hkv
    out, mag, far = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, dl = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        for g in range(Hq):
            at = c.keys(b, g // G, idx, tail_lo)
            for i in range(Mq):
                see = at[at <= c.lens[b] - Mq + i]
                if not len(see):
                    continue
                k, v = c.rows(0, b, g // G, see), c.rows(1, b, g // G, see)
                x = scale * (k @ q[b, g, i])
                m = x.max()
                e = np.exp(x - m)
                z = e.sum()
                p = e / z
                out[b, g, i], mag[b, g, i], far[b, g, i] = p @ v, p @ np.abs(v), np.abs(v).sum(0)
                lse[b, g, i] = m + np.log(z)
                dl[b, g, i] = abs(scale) * (np.abs(k) @ np.abs(q[b, g, i])).max()
    return out, lse, mag, dl, far


def importance(c, q, lse, scale, lo, hi):
    """fx_paged_importance in 64 bits, for the lse given: [B, Hkv, hi - lo], and the largest dl as in attend()."""
    q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
    B, Hq, Mq, _ = q.shape
    G = Hq // c.Hkv
    s = np.zeros((B, c.Hkv, hi - lo))
    dl = 0.0
    for b in range(B):
        for g in range(Hq):
            for i in range(Mq):
                at = np.arange(lo, max(lo, min(hi, c.lens[b] - Mq + i + 1)))
                if not len(at) or lse[b, g, i] == -np.inf:
                    continue
                k = c.rows(0, b, g // G, at)
                s[b, g // G, at - lo] += np.exp(scale * (k @ q[b, g, i]) - lse[b, g, i])
                dl = max(dl, abs(scale) * (np.abs(k) @ np.abs(q[b, g, i])).max() + abs(lse[b, g, i]))
    return s, dl
