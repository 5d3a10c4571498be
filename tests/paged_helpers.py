"""Inputs and plain 64-bit references of the paged-cache tests."""
import math

import numpy as np

from oracle import q64


class Paged:
    """A pool, its table and a ragged batch as numpy arrays.  Everything no
    token owns (pages without an owner, slots past a sequence's end, buffer rows outside the
    batch) holds poison: NaN, or 4-bit metadata of NaN."""

    def __init__(self, bits, heads, kv_heads, d, page, new, past, seed=0, front=0, pad=0, spare=2, share=0):
        rng = np.random.default_rng(seed)
        self.rng, self.bits, self.heads, self.kv_heads, self.d, self.page = rng, bits, heads, kv_heads, d, page
        self.new, self.past = list(new), list(past)
        self.b = len(new)
        self.lens = [n + p for n, p in zip(new, past)]
        per = [-(-x // page) for x in self.lens]
        self.pages = sum(per) + spare
        order = rng.permutation(self.pages)
        self.table_ld = max(per + [1]) + 1
        self.table = np.full((self.b, self.table_ld), -7, np.int32)  # unused entries are no pages
        at = 0
        for i, p in enumerate(per):
            self.table[i, :p] = order[at:at + p]
            at += p
            if i and share:  # a common prefix of read-only pages
                k = min(share, self.past[i] // page, self.past[0] // page)
                self.table[i, :k] = self.table[0, :k]
        self.row_start = (np.cumsum([0] + list(new)) + front).astype(np.int32)
        self.rows = int(self.row_start[-1]) + pad
        self.kv_len = np.array(self.lens, np.int32)
        shape = (self.pages, kv_heads, page)
        self.used = np.zeros((self.pages, page), bool)
        for i in range(self.b):
            for p in range(self.lens[i]):
                self.used[self.table[i, p // page], p % page] = True
        spread = 10.0 ** rng.uniform(-1, 0.3, size=shape + (1,))
        k = (rng.standard_normal(shape + (d,)) * spread).astype(np.float16)
        v = (rng.standard_normal(shape + (d,)) + 0.3 * rng.standard_normal(shape + (1,))).astype(np.float16)
        if bits == 16:
            m = ~np.broadcast_to(self.used[:, None, :], shape)
            k[m], v[m] = np.nan, np.nan
            self.k, self.v, self.km, self.vm = k, v, None, None
        else:
            self.k, self.km = self._codes(k)
            vc, self.vm = self._codes(v)
            self.v = canonical_to_words(vc)
            m = ~np.broadcast_to(self.used[:, None, :], shape)
            self.km[m], self.vm[m] = np.nan, np.nan

    def _codes(self, x):
        codes, mn, sc = q64.quantize(x.reshape(-1))
        s = x.shape
        return (np.asarray(codes).reshape(s[:-1] + (s[-1] // 2,)).copy(),
                np.stack([np.asarray(mn), np.asarray(sc)], -1).reshape(s[:-1] + (s[-1] // 64, 2)).astype(np.float16))

    def where(self, i, p):
        return self.table[i, p // self.page], p % self.page

    def history(self, i, k=None, v=None, km=None, vm=None):
        """Cached keys and values of sequence i as doubles [len][kv_heads][d]."""
        k = self.k if k is None else k
        v = self.v if v is None else v
        km = self.km if km is None else km
        vm = self.vm if vm is None else vm
        p = np.arange(self.lens[i])
        pg, sl = self.table[i, p // self.page], p % self.page
        if self.bits == 16:
            return k[pg, :, sl].astype(np.float64), v[pg, :, sl].astype(np.float64)
        kc = k[pg, :, sl]
        kc = np.stack([kc & 15, kc >> 4], -1).reshape(kc.shape[:-1] + (self.d,))
        vw = v.view(np.uint32)[pg, :, sl // 8]
        vc = (vw >> (4 * (sl % 8)).astype(np.uint32)[:, None, None]) & 15

        def value(c, m):
            m = m[pg, :, sl].astype(np.float32)
            x = c.astype(np.float32).reshape(c.shape[:-1] + (self.d // 64, 64))
            x = (x * m[..., 1:]).astype(np.float32) + m[..., :1]
            return x.astype(np.float16).astype(np.float64).reshape(c.shape)
        return value(kc, km), value(vc, vm)

    def new_rows(self, scale=1.0):
        """K, V and Q rows for the batch, NaN outside it."""
        out = []
        for width in (self.kv_heads * self.d, self.kv_heads * self.d, self.heads * self.d):
            x = (self.rng.standard_normal((self.rows, width)) * scale).astype(np.float16)
            x[: self.row_start[0]] = np.nan
            x[self.row_start[-1]:] = np.nan
            out.append(x)
        return out

    def row_of(self, i, t):
        return int(self.row_start[i]) + t

    def position(self, i, t):
        return self.past[i] + t


def canonical_to_words(codes):
    """Canonical codes [pages][heads][page][d/2] -> token-interleaved words (int32)."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.uint32)
    pg, h, ps, d = c.shape
    c = c.reshape(pg, h, ps // 8, 8, d)
    w = np.zeros((pg, h, ps // 8, d), np.uint32)
    for t in range(8):
        w |= c[:, :, :, t] << np.uint32(4 * t)
    return w.view(np.int32)


def rotate(x, pos, cos_sin, rot, interleaved):
    """fp16 row [heads][d] rotated as documented: fp32 operations, fp16 result."""
    y = x.astype(np.float32).copy()
    c, s = cos_sin[pos, : rot // 2], cos_sin[pos, rot // 2:]
    a = y[:, 0:rot:2].copy() if interleaved else y[:, : rot // 2].copy()
    b = y[:, 1:rot:2].copy() if interleaved else y[:, rot // 2:rot].copy()
    ra, rb = a * c - b * s, b * c + a * s
    if interleaved:
        y[:, 0:rot:2], y[:, 1:rot:2] = ra, rb
    else:
        y[:, : rot // 2], y[:, rot // 2:rot] = ra, rb
    return y.astype(np.float16)


def rope_table(max_pos, rot):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(max_pos)[:, None] * f[None]
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def append_reference(pg: Paged, k, v, q=None, cos_sin=None, rot=0, interleaved=0):
    """The pools (and rotated queries) an append leaves, element by element."""
    pools = [None if x is None else x.copy() for x in (pg.k, pg.v, pg.km, pg.vm)]
    q_out = None if q is None else np.full_like(q, np.nan)
    for i in range(pg.b):
        for t in range(pg.new[i]):
            r, p = pg.row_of(i, t), pg.position(i, t)
            pid, sl = pg.where(i, p)
            kr, vr = k[r].reshape(pg.kv_heads, pg.d), v[r].reshape(pg.kv_heads, pg.d)
            if rot:
                kr = rotate(kr, p, cos_sin, rot, interleaved)
                if q is not None:
                    q_out[r] = rotate(q[r].reshape(pg.heads, pg.d), p, cos_sin, rot, interleaved).reshape(-1)
            if pg.bits == 16:
                pools[0][pid, :, sl], pools[1][pid, :, sl] = kr, vr
                continue
            kc, km = pg._codes(kr)
            vc, vm = pg._codes(vr)
            pools[0][pid, :, sl], pools[2][pid, :, sl], pools[3][pid, :, sl] = kc, km, vm
            codes = np.stack([vc & 15, vc >> 4], -1).reshape(pg.kv_heads, pg.d).astype(np.uint32)
            w = pools[1].view(np.uint32)
            sh = np.uint32(4 * (sl % 8))
            w[pid, :, sl // 8] = (w[pid, :, sl // 8] & ~(np.uint32(15) << sh)) | (codes << sh)
    return pools, q_out


def attention_reference(pg: Paged, q, i, **pools):
    """Rows of sequence i in 64 bits, and the bound each element is held to.

    The bound counts, for a result o = sum p v with weights p (sum 1):
    * the output's rounding, 2^-11 |o| (and half the fp16 subnormal step);
    * the weights' rounding to fp16 before the product, 2^-11 sum p |v|, and for
      weights below fp16's normal range 2^-25 of the row's largest each:
      2^-25 * n max|v| for n keys (the row sum is at least the largest weight);
    * a score's error e (fp32 products and sums over d terms in any order, and the
      scale: (d + 4) 2^-23 of sum |q k| / sqrt d), which changes a weight by a
      factor within 1 +- 2 e, as do exp2's 2^-21 and its argument's rounding,
      2^-23 of the score's own size; the weight sum's error is the same again;
    * fp32 sums over the keys, at most (n / 16 + 40) 2^-23 sum p |v| as tiles of
      16 keys and more are summed by turns.
    """
    kh, vh = pg.history(i, **pools)
    g = pg.heads // pg.kv_heads
    n = pg.new[i]
    out = np.zeros((n, pg.heads, pg.d))
    tol = np.zeros_like(out)
    for j in range(pg.heads):
        kk, vv = kh[:, j // g], vh[:, j // g]
        qq = q[pg.row_start[i]:pg.row_start[i] + n, j * pg.d:(j + 1) * pg.d].astype(np.float64)
        s = qq @ kk.T / math.sqrt(pg.d)
        sa = np.abs(qq) @ np.abs(kk).T / math.sqrt(pg.d)
        mask = np.arange(len(kk))[None] > (pg.past[i] + np.arange(n))[:, None]
        s[mask] = -np.inf
        sa[mask] = 0
        p = np.exp(s - s.max(1, keepdims=True))
        l = p.sum(1, keepdims=True)
        p /= l
        o, a = p @ vv, p @ np.abs(vv)
        e = (pg.d + 4) * 2.0 ** -23 * sa.max(1) + 2.0 ** -21 + 2.0 ** -22 * sa.max(1)
        keys = (~mask).sum(1)
        rel = 2.0 ** -11 + 4 * e + (keys / 16 + 40) * 2.0 ** -23
        vmax = np.abs(vv).max()
        out[:, j] = o
        tol[:, j] = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + rel[:, None] * a + (2.0 ** -25 * keys * vmax)[:, None] / l
    return out.reshape(n, -1), tol.reshape(n, -1)
