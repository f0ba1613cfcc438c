"""Plain forms of the cache in 4 bits, written from the definitions in
include/qsa_cache.h: the coding, the values that blocks stand for (each looked up
by its place in the layout), and histories whose cache is in 4 bits for the plain
attention of cache_helpers.  numpy only; nothing here calls the library."""
import numpy as np

import cache_helpers as ch

E2M1, INT4 = 4, 5
TOP = {E2M1: 6.0, INT4: 7.0}
_E4M3 = ch.e4m3_table()


def e2m1_table():
    """The value of each of the 16 e2m1 codes, from the format's definition."""
    t = np.empty(16)
    for c in range(16):
        s, e, m = c >> 3, (c >> 1) & 3, c & 1
        t[c] = (-1 if s else 1) * (m / 2.0 if e == 0 else (1 + m / 2.0) * 2.0 ** (e - 1))
    return t


def nearest(y, fmt):
    """The code (as a number) nearest to y, the one with an even last bit on ties, at most the largest."""
    y = np.asarray(y, np.float64)
    if fmt == INT4:
        return np.clip(np.rint(y), -7, 7)
    t = e2m1_table()[:8]
    m = np.minimum(np.abs(y), 6.0)
    hi = np.searchsorted(t, m)                     # t[hi - 1] < m <= t[hi]
    lo = np.maximum(hi - 1, 0)
    up = (m - t[lo] > t[hi] - m) | ((m - t[lo] == t[hi] - m) & (hi % 2 == 0))
    return np.copysign(np.where(up, t[hi], t[lo]), y)


def nearest_e4m3(x):
    """x >= 0 rounded to an e4m3 number, ties to even, at most 448."""
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(x, 2.0 ** -40))), -6) - 3)
    return np.rint(x / step) * step


def encode(x, fmt):
    """(codes as numbers, tile scales, scale f32) of x [..., 4, d] f32: products and quotients are binary32's."""
    x = np.asarray(x, np.float32)
    top, f32 = np.float32(TOP[fmt]), np.float32
    with np.errstate(all="ignore"):
        finite = np.isfinite(x).all(axis=(-2, -1))
        z = np.where(finite[..., None, None], x, f32(0))
        amax = np.abs(z).max(axis=(-2, -1))
        s = (amax * f32(1.0 / (448.0 * TOP[fmt]))).astype(f32)
        s = np.where(s >= f32(2.0) ** -126, s, f32(0))
        most = np.abs(z).reshape(*z.shape[:-1], z.shape[-1] // 4, 4).max(axis=(-3, -1))
        unit = (s * top).astype(f32)[..., None]
        q = np.where(unit > 0, most / np.where(unit > 0, unit, f32(1)), f32(0)).astype(f32)
        t = nearest_e4m3(q)
        ts = (t.astype(f32) * s[..., None]).astype(f32)
        by = np.repeat(ts, 4, axis=-1)[..., None, :]
        y = np.where(by > 0, z / np.where(by > 0, by, f32(1)), f32(0)).astype(f32)
        code = np.where(np.repeat(t, 4, axis=-1)[..., None, :] > 0, nearest(y, fmt), 0.0)
    return code, t, np.where(finite, s, f32(np.nan)).astype(f32)


def unpack(blocks, d, fmt):
    """(K, V, tile scales of K, of V) as numbers from blocks [..., 9d/2] (bytes): codes [..., 4, d], scales [..., d/4]."""
    b = blocks.astype(np.int64)
    token, dim = np.arange(4)[:, None], np.arange(d)[None]
    j, c, w, e = dim // 64, dim % 64 // 16, dim % 16 // 8, dim % 8
    word = 128 * j + 64 * (token % 2) + 16 * c + 8 * (token // 2) + 4 * w
    p, second = e % 4, e // 4
    kbit = 8 * p + 4 * second if fmt == E2M1 else 4 * p + 16 * second
    k = (b[..., word + kbit // 8] >> (kbit % 8)) & 15
    m, n, h, w = dim // 64, dim % 64 // 32, dim % 32 // 4, dim % 4 // 2
    word = 2 * d + 128 * m + 16 * h + 8 * n + 4 * w
    p, second = 2 * (dim % 2) + token // 2, token % 2
    vbit = 8 * p + 4 * second if fmt == E2M1 else 4 * p + 16 * second
    v = (b[..., word + vbit // 8] >> (vbit % 8)) & 15
    r = 4 * np.arange(d // 4)
    kt = _E4M3[b[..., 4 * d + r % 64 // 16 * (d // 16) + 4 * (r // 64) + r % 16 // 4]]
    vt = _E4M3[b[..., 4 * d + d // 4 + r % 32 // 4 * (d // 32) + r // 32]]
    if fmt == E2M1:
        t = e2m1_table()
        return t[k], t[v], kt, vt
    return k - 8.0, v - 8.0, kt, vt


class History(ch.History):
    """ch.History with a cache in 4 bits."""

    def coded(self):
        ks, vs = [], []
        for h, t in enumerate(self._lens):
            n = t // 4
            for src, dst in ((self.k, ks), (self.v, vs)):
                x = src[self._tok[h]:self._tok[h] + 4 * n].reshape(n, 4, self.kv_heads, self.d).transpose(0, 2, 1, 3)
                c, t4, s = encode(x, self.fmt)
                dst.append(c * np.repeat(t4, 4, axis=-1)[..., None, :] * s.astype(np.float64)[..., None, None])
        z = np.zeros((0, self.kv_heads, 4, self.d))
        return np.concatenate(ks + [z]), np.concatenate(vs + [z])

    def set_cache(self):
        self.k_cache[self.slot_map], self.v_cache[self.slot_map] = self.k, self.v


def device(h, **kw):
    """ch.device(h) with blocks of 4 bits."""
    import torch
    from top_group_sparse_gb300 import qsa
    t = ch.device(h, **kw)
    t["codes"] = torch.zeros(h.num_blocks, h.kv_heads, 9 * h.d // 2, dtype=torch.uint8, device="cuda")
    t["cache"] = qsa.QsaCodedCache.of(t["codes"], t["scales"], t["block_map"], t["group_offset"], h.fmt)
    return t
