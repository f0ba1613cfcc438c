"""Plain form in 64 bits of what qsa_append_tokens writes (include/qsa_rows.h), and the
batches its tests share.  numpy only; nothing here calls the library."""
import numpy as np

KINDS = ("q", "k", "v", "q_idx", "idx_key")
HALVES, NEIGHBOURS = 0, 1
TWO_PI = 6.283185307179586476925286766559  # of a difference of a few turns: binary64 is enough


def angles(positions, freq):
    """[B, pairs] radians modulo a turn of positions [axes, B] (int) and freq [axes, pairs] f32: the products
    in integers, freq = m * 2^e, against 2 pi to 2^-140."""
    two_pi = 6283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136
    scale = 10 ** 99
    pairs = freq.shape[1]
    out = np.zeros((positions.shape[1], pairs))
    for j in range(pairs):
        parts = []
        for a in range(freq.shape[0]):
            m, e = np.frexp(np.float64(freq[a, j]))
            parts.append((int(m * 2 ** 24), int(e) - 24))
        low = min(e for _, e in parts)
        low = min(low, 0)
        unit = 2 ** -low
        for b in range(positions.shape[1]):
            n = sum(int(positions[a, b]) * m * 2 ** (e - low) for a, (m, e) in enumerate(parts))  # angle = n / unit
            turn = two_pi * unit                      # a turn, in units of 1 / (unit * scale)
            r = (n * scale) % turn
            if 2 * r > turn:
                r -= turn
            out[b, j] = (r * 10 ** 30 // turn) / 1e30 * TWO_PI
    return out


class Batch:
    """Host arrays of one call: a projection per kind in one fused row, where each token goes, positions."""

    def __init__(self, visible, *, q_heads, kv_heads, head_dim, idx_heads, idx_dim, seed, given=KINDS, norms=True,
                 dims=None, idx_dims=None, pairing=HALVES, idx_pairing=None, axes=1, shared=False, eps=1e-5, pad=0,
                 values=None, far=1 << 20):
        r = np.random.RandomState(seed)
        self.visible = np.asarray(visible, np.int32)
        self.B = B = len(visible)
        self.q_heads, self.kv_heads, self.d, self.idx_heads, self.idx_dim = q_heads, kv_heads, head_dim, idx_heads, idx_dim
        self.given, self.eps, self.axes = given, eps, axes
        self.heads = {"q": q_heads, "k": kv_heads, "v": kv_heads, "q_idx": idx_heads, "idx_key": 1}
        self.width = {"q": head_dim, "k": head_dim, "v": head_dim, "q_idx": idx_dim, "idx_key": idx_dim}
        size = {k: self.heads[k] * self.width[k] for k in KINDS}
        self.fused = (r.randn(B, sum(size.values()) + pad) * np.exp(r.randn(B, 1))).astype(np.float32)
        if values is not None:
            self.fused[:] = values(r, self.fused.shape)
        at = np.cumsum([0] + [size[k] for k in KINDS])
        self.slice = {k: slice(int(at[i]), int(at[i + 1])) for i, k in enumerate(KINDS)}
        self.norm = {k: (1 + 0.3 * r.randn(self.width[k])).astype(np.float32) if norms and k != "v" else None for k in KINDS}
        self.turn = {}
        for name, n in (("turn", head_dim if dims is None else dims), ("turn_idx", idx_dim if idx_dims is None else idx_dims)):
            f = 10000.0 ** (-2.0 * np.arange(n // 2) / max(n, 1))
            self.turn[name] = np.stack([np.where(np.arange(n // 2) % axes == a, f, 0.25 * f * (a == 0)) for a in range(axes)]).astype(np.float32)
        self.pairing = {"turn": pairing, "turn_idx": pairing if idx_pairing is None else idx_pairing}
        self.positions = r.randint(-5, far, (axes, B)).astype(np.int32)
        lens = [max(int(max(visible)), 1)] if shared else [max(int(t), 1) for t in visible]
        off = np.concatenate([[0], np.cumsum(lens)])
        self.offset = (np.zeros(B) if shared else off[:-1]).astype(np.int64)
        self.total = int(off[-1])
        self.num_slots = self.total + 7
        self.slot_map = r.permutation(self.num_slots)[:self.total].astype(np.int32)

    def values(self, type_name):
        """The projections as the type holds them, in f32."""
        import torch
        t = torch.from_numpy(self.fused)
        if type_name != "f32":
            t = t.to(torch.bfloat16 if type_name == "bf16" else torch.float16).to(torch.float32)
        return t.numpy()

    def expected(self, type_name):
        """{kind: (rows [B, heads, width] in 64 bits, tolerance of each)}.

        Tolerance (derivation): the sum of a head's squares is off by at most 12 roundings of 2^-24 (three
        products and sums in the lane's pairs, one across, four or five across lanes), its root by half that
        and rsqrt's own 2 * 2^-24 (it is accurate to 2 units in the last place), eps's sum and the product
        with 1/width by 2^-24; two products follow: 12 * 2^-24 in all, 2^-20.  A rotation is two products and
        a sum, 2^-24 of each product and of the sum, of sines and cosines off by 2^-22: with |y_i| + |y_k| as
        the measure, 6 * 2^-24, so 2^-20 + 2^-21 covers both.  Unnormed, unturned values are exact."""
        x = self.values(type_name).astype(np.float64)
        ang = {n: angles(self.positions, f) if f.shape[1] else None for n, f in self.turn.items()}
        out = {}
        for kind in self.given:
            W = self.width[kind]
            y = x[:, self.slice[kind]].reshape(self.B, -1, W)
            tol = np.zeros_like(y)
            if self.norm[kind] is not None:
                y = y / np.sqrt((y ** 2).mean(axis=2, keepdims=True) + np.float64(np.float32(self.eps))) * self.norm[kind]
                tol = 2.0 ** -20 * np.abs(y)
            name = None if kind == "v" else "turn" if kind in ("q", "k") else "turn_idx"
            if name and ang[name] is not None:
                h = ang[name].shape[1]
                one, two = (slice(0, h), slice(h, 2 * h)) if self.pairing[name] == HALVES else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
                c, s = np.cos(ang[name])[:, None], np.sin(ang[name])[:, None]
                a, b = y[..., one].copy(), y[..., two].copy()
                y = y.copy()
                y[..., one], y[..., two] = a * c - b * s, a * s + b * c
                tol[..., one] = tol[..., two] = (2.0 ** -20 + 2.0 ** -21) * (np.abs(a) + np.abs(b))
            out[kind] = (y, tol)
        return out

    def on_device(self, type_name="f32", align=32):
        """A dict of tensors, dims, inputs and tokens; outputs are filled with -9, and start `align` bytes
        into a 256-byte block where that is less than 32."""
        import torch
        from top_group_sparse_gb300 import qsa

        def put(a):
            return torch.from_numpy(np.ascontiguousarray(a)).cuda()

        def room(*shape):
            n = int(np.prod(shape))
            return torch.full((n + 64,), -9.0, device="cuda")[align // 4:align // 4 + n].view(shape)

        t = {"fused": put(self.fused).to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[type_name]),
             "visible": put(self.visible), "positions": put(self.positions), "slot_map": put(self.slot_map),
             "offset": put(self.offset), "q": room(self.B, self.q_heads, self.d), "q_idx": room(self.B, self.idx_heads, self.idx_dim),
             "k_cache": room(self.num_slots, self.kv_heads, self.d), "v_cache": room(self.num_slots, self.kv_heads, self.d),
             "idx_keys": room(self.total, self.idx_dim), "ws": torch.zeros(256, dtype=torch.uint8, device="cuda")}
        t["norm"] = {k: None if v is None else put(v) for k, v in self.norm.items()}
        t["freq"] = {n: put(f) for n, f in self.turn.items()}
        t["dims"] = qsa.make_dims(self.B, self.idx_heads, self.idx_dim, self.q_heads, self.kv_heads, self.d,
                                  max_visible=int(self.visible.max(initial=0)))
        ptr = {k: t[k].data_ptr() for k in ("visible", "q", "q_idx", "idx_keys", "k_cache", "v_cache", "slot_map")}
        t["inputs"] = qsa.QsaInputs(num_slots=self.num_slots, key_offset=t["offset"].data_ptr(),
                                    slot_offset=t["offset"].data_ptr(), **ptr)
        t["tokens"] = qsa.QsaNewTokens.of(
            **{k: t["fused"][:, self.slice[k]] for k in self.given}, positions=t["positions"], freq=t["freq"]["turn"],
            idx_freq=t["freq"]["turn_idx"], pairing=self.pairing["turn"], idx_pairing=self.pairing["turn_idx"], eps=self.eps,
            **{k + "_norm": t["norm"][k] for k in self.given if k != "v"})
        return t

    def places(self):
        """The rows of the caches that the tokens go to, of the queries that have one."""
        has = self.visible > 0
        row = self.offset[has] + self.visible[has] - 1
        return has, row, self.slot_map[row]

    def check(self, t, type_name="f32"):
        """Every output of the call on `t`: the tokens' rows within their tolerances, all others untouched."""
        want = self.expected(type_name)
        has, row, slot = self.places()
        spot = {"q": ("q", np.flatnonzero(has)), "q_idx": ("q_idx", np.flatnonzero(has)), "k": ("k_cache", slot),
                "v": ("v_cache", slot), "idx_key": ("idx_keys", row)}
        for kind, (name, at) in spot.items():
            got = t[name].cpu().numpy().reshape(t[name].shape[0], -1, self.width[kind])
            left = np.ones(len(got), bool)
            if kind in self.given:
                left[at] = False
                y, tol = want[kind]
                err = np.abs(got[at].astype(np.float64) - y[has])
                assert (err <= tol[has]).all(), (kind, float((err - tol[has]).max()))
            assert (got[left] == -9).all(), kind
