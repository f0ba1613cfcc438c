"""Plain forms in 64 bits of the coded cache, the attention over it and the
eviction, and the workloads their tests share.  numpy only, written from the
definitions in include/qsa_cache.h; nothing here calls the library."""
import numpy as np

QMAX = {0: 448.0, 1: 127.0}  # by format: e4m3, int8
E4M3, INT8 = 0, 1


def e4m3_table():
    """The value of each of the 256 e4m3 codes, from the format's definition."""
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = np.nan if (e == 15 and m == 7) else (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
        t[c] = -v if s else v
    return t


_TABLE = e4m3_table()


def code_values(raw, fmt):
    """The numbers that code bytes stand for."""
    return _TABLE[raw] if fmt == E4M3 else raw.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """(codes as numbers, scale f32) of x [..., 4, d] f32 over its last two axes."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        finite = np.isfinite(x).all(axis=(-2, -1))
        amax = np.abs(np.where(np.isfinite(x), x, 0)).max(axis=(-2, -1)).astype(np.float32)
        s = (amax * (np.float32(1) / np.float32(QMAX[fmt]))).astype(np.float32)
        s = np.where(s >= np.float32(2.0) ** -126, s, np.float32(0))
        y = np.where((s > 0)[..., None, None] & finite[..., None, None], x / np.where(s > 0, s, 1)[..., None, None].astype(np.float32), 0)
    y = y.astype(np.float64)
    if fmt == INT8:
        c = np.clip(np.rint(y), -127, 127)
    else:
        e = np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -60))), -6)
        step = 2.0 ** (e - 3)
        c = np.clip(np.rint(y / step) * step, -448, 448)
    return c, np.where(finite, s, np.float32(np.nan)).astype(np.float32)


def unpack(codes, d, fmt):
    """K, V [n, kv, 4, d] as numbers from the blocks [n, kv, 8d] of a cache."""
    n, kv = codes.shape[:2]
    k = codes[:, :, :4 * d].reshape(n, kv, d // 64, 4, 64).transpose(0, 1, 3, 2, 4).reshape(n, kv, 4, d)
    v = codes[:, :, 4 * d:].reshape(n, kv, d, 4).transpose(0, 1, 3, 2)
    return code_values(np.ascontiguousarray(k), fmt), code_values(np.ascontiguousarray(v), fmt)


class History:
    """Host arrays of a batch with a coded cache: every complete group coded in
    a permuted block, the raw tails in a small f32 cache."""

    def __init__(self, visible, *, q_heads, kv_heads, head_dim, fmt, seed, shared=False, spare_blocks=3, q_scale=1.0,
                 idx_dim=64):
        r = np.random.RandomState(seed)
        self.visible = np.asarray(visible, np.int32)
        self.B, self.q_heads, self.kv_heads, self.d, self.fmt = len(visible), q_heads, kv_heads, head_dim, fmt
        self.shared, self.idx_dim = shared, idx_dim
        lens = [int(max(visible))] if shared else [int(t) for t in visible]
        tok = np.concatenate([[0], np.cumsum(lens)])
        grp = np.concatenate([[0], np.cumsum([t // 4 for t in lens])])
        wgt = np.concatenate([[0], np.cumsum([-(-t // 4) for t in lens])])
        pick = np.zeros(self.B, np.int64) if shared else np.arange(self.B)
        self.token_offset = tok[pick].astype(np.int64)
        self.group_offset = grp[pick].astype(np.int64)
        self.weight_offset = wgt[pick].astype(np.int64)
        total, groups = int(tok[-1]), int(grp[-1])
        self.n_weights = int(wgt[-1])
        self.k = r.randn(max(total, 1), kv_heads, head_dim).astype(np.float32)
        self.v = r.randn(max(total, 1), kv_heads, head_dim).astype(np.float32)
        self.q = (r.randn(self.B, q_heads, head_dim) * q_scale).astype(np.float32)
        self.num_slots = total + 5
        self.slot_map = r.permutation(self.num_slots)[:max(total, 1)].astype(np.int32)
        self.k_cache = np.full((self.num_slots, kv_heads, head_dim), 7.0, np.float32)
        self.v_cache = np.full((self.num_slots, kv_heads, head_dim), 7.0, np.float32)
        self.k_cache[self.slot_map], self.v_cache[self.slot_map] = self.k, self.v
        self.num_blocks = groups + spare_blocks
        self.block_map = r.permutation(self.num_blocks)[:max(groups, 1)].astype(np.int32)
        self.scale = float(np.float32(1.0 / np.sqrt(head_dim)))
        self._grp, self._lens = grp, lens
        self._tok = tok
        self.weights0 = (r.rand(max(self.n_weights, 1)) * 4).astype(np.float32)

    def group_ranges(self):
        """(begin, end) per query that code every complete group of every history once."""
        end = self.visible // 4
        if self.shared:
            own = np.arange(self.B) == int(np.argmax(self.visible))
            end = np.where(own, end, 0)
        return np.zeros(self.B, np.int32), end.astype(np.int32)

    def coded(self):
        """Values (f64) of the coded rows of every history's complete groups, by global group."""
        ks, vs = [], []
        for h, t in enumerate(self._lens):
            n = t // 4
            for src, dst in ((self.k, ks), (self.v, vs)):
                x = src[self._tok[h]:self._tok[h] + 4 * n].reshape(n, 4, self.kv_heads, self.d).transpose(0, 2, 1, 3)
                c, s = encode(x, self.fmt)
                dst.append(c * s.astype(np.float64)[..., None, None])
        z = np.zeros((0, self.kv_heads, 4, self.d))
        return np.concatenate(ks + [z]), np.concatenate(vs + [z])


def attention(h, rows=None, coded=None):
    """(out, weight shares by query, tolerance of out) in 64 bits.  rows: the ID
    row of each query (None: every visible token).  coded: the coded rows'
    values (K, V), by default those of the plain coding.

    Tolerance, relative to max|V| (derivation): with S = scale * max_t
    sum_j |q_j k_tj|, a score is off by at most 7 * 2^-22 * S -- q's two 16-bit
    parts leave 2^-22, the eight accumulations of a chain, truncated, 8 * 2^-23,
    the products with the scales 3 * 2^-24, the rounding of the exponential's
    argument 2^-24 of it -- and the output by twice that; the weights' two parts
    and the exponential leave 2 * 2^-22, the accumulations of the second product
    and the additions over at most 16 steps, 8 warps and 64 runs' slices (each
    half a step, 2^-24) 28 * 2^-22 more."""
    K, V = h.coded() if coded is None else coded
    out = np.zeros((h.B, h.q_heads, h.d))
    share, tol, xs = [], np.zeros(h.B), []
    r = h.q_heads // h.kv_heads
    for b in range(h.B):
        T = int(h.visible[b])
        row = np.arange(T) if rows is None else np.asarray(rows[b], np.int64)
        n = len(row) // 4 * 4
        g, tail = row[:n:4] // 4, row[n:]
        w = np.zeros(-(-T // 4))
        S = vmax = 0.0
        for kv in range(h.kv_heads):
            kk = np.concatenate([K[h.group_offset[b] + g, kv].reshape(-1, h.d),
                                 h.k[h.token_offset[b] + tail, kv].astype(np.float64)])
            vv = np.concatenate([V[h.group_offset[b] + g, kv].reshape(-1, h.d),
                                 h.v[h.token_offset[b] + tail, kv].astype(np.float64)])
            if len(row) == 0:
                continue
            q = h.q[b, kv * r:(kv + 1) * r].astype(np.float64)
            x = (q @ kk.T) * h.scale
            S = max(S, float((np.abs(q) @ np.abs(kk).T).max()) * h.scale)
            vmax = max(vmax, float(np.abs(vv).max()))
            p = np.exp(x - x.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            out[b, kv * r:(kv + 1) * r] = p @ vv
            np.add.at(w, row // 4, p.sum(axis=0))
        share.append(w)
        tol[b] = vmax * 2.0 ** -22 * (14 * S + 30)
        xs.append(2.0 ** -22 * (14 * S + 30))
    return out, share, tol, xs


def add_weights(h, share, rel):
    """(accumulators, tolerance): the queries' shares added to weights0.  A share
    is off by its relative tolerance, a sum by half a step of each addition
    (queries of one history) and of the at most 16 heads'."""
    w = h.weights0.astype(np.float64).copy()
    tol = np.zeros_like(w)
    for b in range(h.B):
        at = h.weight_offset[b]
        w[at:at + len(share[b])] += share[b]
        tol[at:at + len(share[b])] += share[b] * (rel[b] + 16 * 2.0 ** -24) + 2.0 ** -24 * w[at:at + len(share[b])]
    return w, tol + 1e-30


def evict(visible, weights, offset, keep, sink, recent):
    """Kept groups of each query, ascending, from the definition."""
    res = []
    for b, T in enumerate(visible):
        G = int(T) // 4
        w = weights[offset[b]:offset[b] + G].astype(np.float64)
        if G <= keep:
            res.append(np.arange(G))
            continue
        mid = np.arange(sink, G - recent)
        nan = np.isnan(w[mid])
        order = np.lexsort((mid, np.where(nan, 0, -np.where(nan, 0, w[mid])), nan))
        best = mid[order[:keep - sink - recent]]
        res.append(np.sort(np.concatenate([np.arange(sink), best, np.arange(G - recent, G)])).astype(np.int64))
    return res


# ---- on the GPU ------------------------------------------------------------------

def device(h, budget=512, whole=False, weights=False, idx_heads=8, max_visible=None):
    """The history's arrays in device memory, with dims, inputs, cache, outputs and
    a workspace: a dict of tensors and of the binding's structures."""
    import torch
    from top_group_sparse_gb300 import qsa

    def put(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    t = {k: put(getattr(h, k)) for k in ("visible", "q", "k_cache", "v_cache", "slot_map", "token_offset", "group_offset",
                                         "weight_offset", "block_map")}
    t["codes"] = torch.zeros(h.num_blocks, h.kv_heads, 8 * h.d, dtype=torch.uint8, device="cuda")
    t["scales"] = torch.zeros(h.num_blocks, h.kv_heads, 2, device="cuda")
    t["weights"] = put(h.weights0)
    t["out"] = torch.full((h.B, h.q_heads, h.d), float("nan"), device="cuda")
    dims = qsa.make_dims(h.B, idx_heads, h.idx_dim, h.q_heads, h.kv_heads, h.d, budget_groups=budget,
                         max_visible=int(h.visible.max(initial=0)) if max_visible is None else max_visible, scale=h.scale)
    t["dims"] = dims
    t["ws"] = torch.zeros(qsa.qsa_coded_workspace_size(dims, whole, weights), dtype=torch.uint8, device="cuda")
    t["inputs"] = qsa.QsaInputs(visible=t["visible"].data_ptr(), q=t["q"].data_ptr(), k_cache=t["k_cache"].data_ptr(),
                                v_cache=t["v_cache"].data_ptr(), num_slots=h.num_slots, slot_map=t["slot_map"].data_ptr(),
                                slot_offset=t["token_offset"].data_ptr())
    t["cache"] = qsa.QsaCodedCache.of(t["codes"], t["scales"], t["block_map"], t["group_offset"], h.fmt)
    lo, hi = h.group_ranges()
    t["lo"], t["hi"] = put(lo), put(hi)
    t["most"] = int((hi - lo).max(initial=0))
    return t


def fill_cache(h, t):
    from top_group_sparse_gb300 import qsa
    qsa.qsa_code_groups(t["dims"], t["inputs"], t["cache"], t["lo"], t["hi"], t["most"], t["ws"])


def rows_to_device(rows, budget):
    import torch
    cap = 4 * budget + 3
    ids = np.full((len(rows), cap), -1, np.int32)
    for b, r in enumerate(rows):
        ids[b, :len(r)] = r
    n = np.array([len(r) for r in rows], np.int32)
    return torch.from_numpy(ids).cuda(), torch.from_numpy(n).cuda()


def some_rows(h, budget, seed):
    """Rows as a selection emits them: up to `budget` random groups ascending, then the tail."""
    r = np.random.RandomState(seed)
    rows = []
    for T in h.visible:
        G = int(T) // 4
        g = np.sort(r.permutation(G)[:budget])
        rows.append(np.concatenate([(4 * g[:, None] + np.arange(4)).ravel(), np.arange(4 * G, int(T))]).astype(np.int64))
    return rows
