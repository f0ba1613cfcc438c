"""Cases of the rows that go into the caches and come back, and of the K/V cache in 4 bits.

Four operators, each with its plain form (elementary torch operations in 32
bits, angles in 64) and the library's call:

* ``append`` -- the new token of every query: its projected rows normalised per
  head, rotated by its position and written where the path reads them
  (``qsa_append_tokens``);
* ``store``  -- complete four-token groups coded in 4 bits (a scale per group and
  KV head, one per tile of four tokens by four dims) and read back as 32-bit rows
  (``qsa_code_groups``, ``qsa_read_groups``);
* ``read``   -- groups of a coded cache, in 4 or in 8 bits, read back as 32-bit
  rows at their slots (``qsa_read_groups``);
* ``attend`` -- attention of one query per batch entry over a cache held in 4
  bits: over every visible token, or over the token rows that a selection
  emitted, with the attention that each group received added to running
  accumulators where the case asks for it (``qsa_attend_coded``).

What is held in 4 or 8 bits is returned as the values it stands for.
"""
import math
import random

import torch

own = False

GROUP = 4
DEV = "cuda"
TOP = {"e4m3": 448.0, "int8": 127.0, "e2m1": 6.0, "int4": 7.0}  # each format's largest code
FORMAT = {"e4m3": 0, "int8": 1, "e2m1": 4, "int4": 5}
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # A decode step of 32 sequences: one token each, from a projection in bf16: latency.
        dict(name="append_step", op="append", batch=32, tokens=2052, kind="equal", heads=16, kv=2, d=128, ih=8, idx=64,
             type="bf16", axes=1, rot=128, idx_rot=64, pairing="halves", norm=True),
        # A chunk of 256 consecutive positions of one history, rotated in part, without norms, in 32 bits.
        dict(name="append_chunk", op="append", batch=256, tokens=100256, kind="shared", heads=16, kv=2, d=128, ih=8, idx=64,
             type="f32", axes=1, rot=64, idx_rot=32, pairing="neighbours", norm=False),
        # A prompt of images or video: 32,768 tokens with positions in time, height and width.
        dict(name="append_prompt", op="append", batch=32768, tokens=32768, kind="shared", heads=16, kv=2, d=128, ih=8, idx=64,
             type="bf16", axes=3, rot=128, idx_rot=64, pairing="halves", norm=True),
        # Every one of 32 sequences completes a group: latency.
        dict(name="store_step", op="store", batch=32, tokens=2052, groups=1, kv=2, d=128, fmt="e2m1"),
        # A prompt's cache coded at once, after a chunked prefill of 100,000 positions.
        dict(name="store_prompt", op="store", batch=1, tokens=100255, groups=25063, kv=2, d=128, fmt="int4"),
        # Eight histories of 65,537 tokens given their last 8,192 back in 32 bits.
        dict(name="read_recent", op="read", batch=8, tokens=65537, groups=2048, kv=2, d=128, fmt="e2m1"),
        # A short history read back from 8 bits: latency.
        dict(name="read_short", op="read", batch=1, tokens=2052, groups=513, kv=2, d=64, fmt="e4m3"),
        # The smallest history: one query, one head, 37 tokens (9 groups and one raw token).
        dict(name="attend4_t37", op="attend", batch=1, tokens=37, kind="equal", rows=0, weights=False,
             heads=1, kv=1, d=64, fmt="int4"),
        # Layers that attend to everything: 8 long sequences.
        dict(name="attend4_long", op="attend", batch=8, tokens=262144, kind="equal", rows=0, weights=False,
             heads=16, kv=2, d=128, fmt="e2m1"),
        # A serving batch of mixed lengths up to 65,537, an empty one and a raw tail alone among them.
        dict(name="attend4_ragged", op="attend", batch=32, tokens=65537, kind="ragged", rows=0, weights=False,
             heads=16, kv=2, d=128, fmt="int4"),
        # The observation pass before an eviction: every token's weight, sixteen query heads on one KV head.
        dict(name="attend4_observe", op="attend", batch=4, tokens=40003, kind="equal", rows=0, weights=True,
             heads=16, kv=1, d=128, fmt="int4"),
        # A chunk of 256 consecutive positions of one history, each with its own selected rows; what
        # they attend to is accumulated for the history that they share.
        dict(name="rows4_chunk", op="attend", batch=256, tokens=100256, kind="shared", rows=512, weights=True,
             heads=16, kv=2, d=128, fmt="e2m1"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "append", "store", "read", "attend", "attend", "attend"])
    heads, kv, d = rng.choice([(1, 1, 64), (2, 2, 64), (8, 8, 64), (8, 2, 64), (16, 2, 128), (16, 1, 128),
                               (32, 8, 128), (12, 4, 128), (10, 2, 128)])
    if op == "append":
        ih, idx = rng.choice([(4, 32), (8, 32), (4, 64), (8, 64)])
        kind = rng.choice(["equal", "ragged", "shared"])
        batch = _log(rng, 1, min(32768, 2 ** 26 // ((heads + 2 * kv) * d + (ih + 1) * idx)))
        tokens = batch + _log(rng, 1, 65536) if kind == "shared" else _log(rng, 1, max(1, 2 ** 18 // batch))
        return dict(op=op, batch=batch, tokens=tokens, kind=kind, heads=heads, kv=kv, d=d, ih=ih, idx=idx,
                    type=rng.choice(["bf16", "bf16", "f16", "f32"]), axes=rng.choice([1, 1, 2, 3, 4]),
                    rot=8 * rng.randrange(0, d // 8 + 1), idx_rot=8 * rng.randrange(0, idx // 8 + 1),
                    pairing=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7)
    if op in ("store", "read"):
        batch = _log(rng, 1, 64)
        groups = _log(rng, 1, 2 ** 15 // (batch * kv))
        tokens = GROUP * (groups + rng.randrange(0, 500)) + rng.randrange(4)
        return dict(op=op, batch=batch, tokens=tokens, groups=groups, kv=kv, d=d,
                    fmt=rng.choice(["e2m1", "int4"] + (["e4m3", "int8"] if op == "read" else [])))
    most = 2 ** 29 // (max(kv, heads // 8) * d)  # tokens in all
    kind = rng.choice(["equal", "ragged", "ragged", "shared"])
    rows = rng.choice([0, 0, 512, _log(rng, 1, 512)])
    if rows:
        batch = _log(rng, 1, 256 if kind == "shared" else 32)
        tokens = _log(rng, 1, min(262144, most // (1 if kind == "shared" else batch)))
    else:  # every query reads its whole history
        batch = _log(rng, 1, 32)
        tokens = _log(rng, 1, min(262144, most // batch))
    return dict(op=op, batch=batch, tokens=max(tokens, batch if kind == "shared" else 1), kind=kind, rows=rows,
                weights=rng.random() < 0.4, heads=heads, kv=kv, d=d, fmt=rng.choice(["e2m1", "int4"]))


def _lengths(c):
    """Visible tokens of each query: a property of the case, whatever the seed."""
    B, T = c["batch"], c["tokens"]
    if c.get("kind") == "ragged":
        r = random.Random("%d %d" % (B, T))
        lens = [T] + [r.randrange(0, T + 1) for _ in range(B - 1)]
        if B >= 4:
            lens[1], lens[2] = 0, min(3, T)
        return lens
    if c.get("kind") == "shared":
        return [T - B + 1 + b for b in range(B)]
    return [T] * B


def _block_bytes(c):
    """Of one (group, KV head), its one scale for K and one for V included."""
    return (9 * c["d"] // 2 if c["fmt"] in ("e2m1", "int4") else 8 * c["d"]) + 8


def work(c):
    if c["op"] == "append":
        n = sum(t > 0 for t in _lengths(c))
        values = (c["heads"] + 2 * c["kv"]) * c["d"] + (c["ih"] + 1) * c["idx"]
        turned = (c["heads"] + c["kv"]) * c["rot"] + (c["ih"] + 1) * c["idx_rot"]
        return {"bytes": n * (values * (4 + TYPE[c["type"]].itemsize) + 4 * c["axes"] + 24),
                "flops": n * (3 * turned + (4 * values if c["norm"] else 0))}
    if c["op"] in ("store", "read"):
        n = c["batch"] * c["groups"]
        rows = 2 * GROUP * c["d"] * 4  # of K and V of one group and head
        moved = rows + _block_bytes(c) if c["op"] == "read" else 2 * rows + _block_bytes(c)
        return {"bytes": n * (c["kv"] * moved + 20), "flops": n * c["kv"] * 2 * GROUP * c["d"] * (2 if c["op"] == "read" else 4)}
    lens = _lengths(c)
    kv, d, nq = c["kv"], c["d"], c["heads"]
    groups = [min(t // GROUP, c["rows"]) if c["rows"] else t // GROUP for t in lens]
    # queries of one history share what they read
    blocks = sum(groups) if c["kind"] != "shared" else min(sum(groups), max(lens) // GROUP)
    tail = sum(t % GROUP for t in lens)
    moved = blocks * (kv * _block_bytes(c) + 4) + tail * kv * d * 8 + len(lens) * nq * d * 8
    if c["rows"]:
        moved += sum(groups) * 16
    if c["weights"]:
        moved += blocks * 8
    return {"bytes": moved, "flops": 4 * nq * d * sum(GROUP * g + t % GROUP for g, t in zip(groups, lens))}


# ---- the coded cache's layout ------------------------------------------------------
# A block in 4 bits: 2d bytes of K, 2d of V, d/4 tile scales of K, d/4 of V.

def _pairs(a, b, fmt):
    """Bytes from the codes a, b of the pairs p = 0..3 (last axis) of each word.  e2m1: pair p is byte p; int4: a of
    pair p is nibble p, b nibble p + 4."""
    if fmt == "e2m1":
        return a | (b << 4)
    n = torch.cat([a, b], dim=-1)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpairs(w, fmt):
    lo, hi = w & 15, w >> 4
    if fmt == "e2m1":
        return lo, hi
    n = torch.stack([lo, hi], dim=-1).flatten(-2)
    return n[..., :4], n[..., 4:]


def _pack4(kn, vn, kt, vt, fmt):
    """Blocks (bytes) of K and V codes [..., 4, d] and their tile scales' bytes [..., d/4]."""
    d, lead = kn.shape[-1], kn.shape[:-2]
    at = range(len(lead))
    k = kn.reshape(*lead, 2, 2, d // 64, 4, 2, 2, 4)      # t, parity, j, chunk, word, half, p: token 2t + parity
    k = k.permute(*at, *(len(lead) + i for i in (2, 1, 3, 0, 4, 5, 6)))
    k = _pairs(k[..., 0, :], k[..., 1, :], fmt).flatten(len(lead))
    v = vn.reshape(*lead, 2, 2, d // 64, 2, 8, 2, 2)      # token pair, token, m, n, h, word, dim
    v = v.permute(*at, *(len(lead) + i for i in (2, 4, 3, 5, 1, 6, 0))).flatten(-2)  # m, h, n, word, token, (dim, pair)
    v = _pairs(v[..., 0, :], v[..., 1, :], fmt).flatten(len(lead))
    kt = kt.reshape(*lead, d // 64, 4, 4).transpose(-3, -2).flatten(len(lead))
    vt = vt.reshape(*lead, d // 32, 8).transpose(-2, -1).flatten(len(lead))
    return torch.cat([k, v, kt, vt], dim=-1).contiguous()


def _unpack4(raw, d, fmt):
    """(K, V) [..., 4, d]: codes times tile scales, in 32 bits (exact)."""
    lead = raw.shape[:-1]
    at = range(len(lead))
    k, v, kt, vt = raw.split([2 * d, 2 * d, d // 4, d // 4], dim=-1)
    k = torch.stack(_unpairs(k.reshape(*lead, d // 64, 2, 4, 2, 2, 4), fmt), dim=-2)       # j, parity, chunk, t, word, half, p
    k = k.permute(*at, *(len(lead) + i for i in (3, 1, 0, 2, 4, 5, 6))).reshape(*lead, 4, d)
    v = torch.stack(_unpairs(v.reshape(*lead, d // 64, 8, 2, 2, 4), fmt), dim=-2)          # m, h, n, word, token, (dim, pair)
    v = v.unflatten(-1, (2, 2)).permute(*at, *(len(lead) + i for i in (6, 4, 0, 2, 1, 3, 5))).reshape(*lead, 4, d)
    f8 = torch.float8_e4m3fn
    kt = kt.contiguous().view(f8).to(torch.float32).reshape(*lead, 4, d // 64, 4).transpose(-3, -2).flatten(-3)
    vt = vt.contiguous().view(f8).to(torch.float32).reshape(*lead, 8, d // 32).transpose(-2, -1).flatten(-2)

    def times(codes, t):
        codes = codes.to(torch.float32)
        if fmt == "int4":
            x = codes - 8
        else:
            m = torch.where(codes >= 8, codes - 8, codes)  # 0 .. 7: 0, .5, 1, 1.5, 2, 3, 4, 6
            m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
            x = torch.where(codes >= 8, -m, m)
        return (x.unflatten(-1, (d // 4, 4)) * t[..., None, :, None]).flatten(-2)

    return times(k, kt), times(v, vt)


def _pack8(kc, vc):
    """8-bit codes of K and V [..., 4, d] in a block's layout: K as [d/64][4][64], V as [d][4]."""
    d = kc.shape[-1]
    k = kc.unflatten(-1, (d // 64, 64)).transpose(-3, -2).flatten(-3)
    return torch.cat([k, vc.transpose(-1, -2).flatten(-2)], dim=-1)


def _decoded(raw, scales, d, fmt):
    """(K, V) [..., 4, d]: the values that blocks [..., bytes] with scales [..., 2] stand for."""
    if fmt in ("e2m1", "int4"):
        k, v = _unpack4(raw, d, fmt)
    else:
        kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
        k = raw[..., :4 * d].unflatten(-1, (d // 64, GROUP, 64)).transpose(-3, -2).contiguous().view(kind).to(torch.float32)
        v = raw[..., 4 * d:].unflatten(-1, (d, GROUP)).transpose(-1, -2).contiguous().view(kind).to(torch.float32)
        k = k.flatten(-2)
    return k * scales[..., 0, None, None], v * scales[..., 1, None, None]


def _to_codes8(x, fmt):
    """8-bit codes (as bytes) and scales of x [..., 4, d] over its last two axes."""
    scale = x.abs().amax(dim=(-2, -1)) / TOP[fmt]
    y = (x / torch.where(scale > 0, scale, 1.0)[..., None, None]).clamp(-TOP[fmt], TOP[fmt])
    code = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(y).to(torch.int8)
    return code.view(torch.uint8), scale


def _to_codes4(x, fmt):
    """4-bit codes, tile scales (e4m3, as bytes) and scales of x [..., 4, d] f32 over its last two axes."""
    top = TOP[fmt]
    amax = x.abs().amax(dim=(-2, -1))
    scale = amax * torch.tensor(1.0 / (448.0 * top), dtype=torch.float32, device=x.device)
    scale = torch.where(scale >= 2.0 ** -126, scale, 0.0)
    tile = x.unflatten(-1, (x.shape[-1] // 4, 4))                     # [..., 4 tokens, tiles, 4 dims]
    most = tile.abs().amax(dim=(-3, -1))
    unit = (scale * top)[..., None]
    t = torch.where(unit > 0, most / torch.where(unit > 0, unit, 1.0), 0.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = t.to(torch.float32) * scale[..., None]
    y = tile / torch.where(s > 0, s, 1.0)[..., None, :, None]
    y = torch.where((s > 0)[..., None, :, None], y, 0.0).clamp(-top, top)
    if fmt == "int4":
        code = torch.round(y).to(torch.int16) + 8
    else:
        m = y.abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        m = torch.round(m / step) * step                              # 0, .5, 1, 1.5, 2, 3, 4, 6 -> 0 .. 7
        m = torch.where(m <= 2, 2 * m, torch.where(m <= 4, m + 2, m / 2 + 4))
        code = m.to(torch.int16) + 8 * torch.signbit(y).to(torch.int16)
    return code.to(torch.uint8).flatten(-2), t.view(torch.uint8), scale


def _to_block(k, v, fmt):
    """Blocks (bytes) and scales [..., 2] of K and V [..., 4, d] f32."""
    if fmt in ("e2m1", "int4"):
        kc, kt, ks = _to_codes4(k, fmt)
        vc, vt, vs = _to_codes4(v, fmt)
        return _pack4(kc, vc, kt, vt, fmt), torch.stack([ks, vs], dim=-1)
    kc, ks = _to_codes8(k, fmt)
    vc, vs = _to_codes8(v, fmt)
    return _pack8(kc, vc), torch.stack([ks, vs], dim=-1)


# ---- inputs ---------------------------------------------------------------------

def _offsets(sizes, shared=False):
    """First row of each query in a packed array of regions of these sizes."""
    if shared:
        return torch.zeros(len(sizes), dtype=torch.int64, device=DEV), max(sizes)
    at, off = 0, []
    for n in sizes:
        off.append(at)
        at += n
    return torch.tensor(off, dtype=torch.int64, device=DEV), at


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    lens = _lengths(c)
    s = {"case": c, "visible": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    s |= {"append": _prepare_append, "attend": _prepare_attend}.get(c["op"], _prepare_groups)(c, lens, s["visible"], gen)
    if own:
        s["plan"] = _plan(s)
    return s


def _prepare_append(c, lens, visible, gen):
    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    B, nq, kv, d, ih, idx = c["batch"], c["heads"], c["kv"], c["d"], c["ih"], c["idx"]
    shared = c["kind"] == "shared"
    s = {}
    s["slot_offset"], total = _offsets(lens, shared)
    total = max(total, 1)
    # one matrix product made a token's rows side by side; a few channels are wide, as trained projections' are
    widths = {"q": nq * d, "k": kv * d, "v": kv * d, "q_idx": ih * idx, "idx_key": idx}
    x = (randn(B, sum(widths.values())) * (1 + 7 * (torch.rand(sum(widths.values()), generator=gen, device=DEV) > 0.97)))
    x = x.to(TYPE[c["type"]])
    s["rows"] = dict(zip(widths, x.split(list(widths.values()), dim=1)))
    # the slots of earlier tokens are others' business
    s["slot_map"] = torch.zeros(total, dtype=torch.int32, device=DEV)
    has = visible > 0
    slots = torch.randperm(2 * B, generator=gen, device=DEV)[:B].to(torch.int32)
    s["slot_map"][(s["slot_offset"] + visible - 1)[has]] = slots[has]
    # positions run ahead of the places in the cache after an eviction
    s["positions"] = torch.zeros(c["axes"], B, dtype=torch.int32, device=DEV)
    ahead = int(torch.randint(0, 1 << 20, (1,), generator=gen, device=DEV))
    s["positions"][0] = visible + ahead
    if c["axes"] > 1:  # height, width, ...: places in a picture
        s["positions"][1:] = torch.randint(0, 2048, (c["axes"] - 1, B), generator=gen, device=DEV).to(torch.int32)
    for name, rot in (("freq", c["rot"]), ("idx_freq", c["idx_rot"])):
        j = torch.arange(rot // 2, device=DEV)
        f = 10000.0 ** (-2.0 * j / max(rot, 1))
        s[name] = torch.stack([torch.where(j % c["axes"] == a, f, 0.0) for a in range(c["axes"])]).to(torch.float32)
    for name, w in (("q_norm", d), ("k_norm", d), ("q_idx_norm", idx), ("idx_key_norm", idx)):
        s[name] = 1 + 0.2 * randn(w) if c["norm"] else None
    s["q"], s["q_idx"] = torch.zeros(B, nq, d, device=DEV), torch.zeros(B, ih, idx, device=DEV)
    s["k_cache"], s["v_cache"] = torch.zeros(2 * B, kv, d, device=DEV), torch.zeros(2 * B, kv, d, device=DEV)
    s["idx_keys"] = torch.zeros(total, idx, device=DEV)
    return s


def _prepare_groups(c, lens, visible, gen):
    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    kv, d = c["kv"], c["d"]
    s = {}
    # a sequence's last `groups` groups are coded or read; its blocks and slots are wherever they were free
    n = c["groups"]
    s["slot_offset"], total = _offsets(lens)
    s["block_offset"], blocks = _offsets([t // GROUP for t in lens])
    end = visible // GROUP
    s["group_begin"], s["group_end"] = (end - n).contiguous(), end.contiguous()
    taken = c["batch"] * n
    pages = -(-taken * GROUP // 16)
    s["slot_map"] = torch.zeros(total, dtype=torch.int32, device=DEV)
    s["block_map"] = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    g = s["group_begin"][:, None] + torch.arange(n, device=DEV)
    s["block_map"][s["block_offset"][:, None] + g] = torch.randperm(taken, generator=gen, device=DEV).to(torch.int32).reshape(-1, n)
    t = torch.arange(taken * GROUP, device=DEV)  # pages of 16 tokens
    slots = (torch.randperm(pages, generator=gen, device=DEV)[t // 16] * 16 + t % 16).to(torch.int32)
    at = s["slot_offset"][:, None, None] + GROUP * g[..., None] + torch.arange(GROUP, device=DEV)
    s["slot_map"][at] = slots.reshape(-1, n, GROUP)
    wide = 1 + 7 * (torch.rand(kv, d, generator=gen, device=DEV) > 0.95)  # keys carry a few wide channels
    s["k_back"], s["v_back"] = torch.zeros(pages * 16, kv, d, device=DEV), torch.zeros(pages * 16, kv, d, device=DEV)
    if c["op"] == "store":
        s["k_cache"], s["v_cache"] = randn(pages * 16, kv, d) * wide, randn(pages * 16, kv, d)
        s["codes"] = torch.zeros(taken, kv, _block_bytes(c) - 8, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(taken, kv, 2, device=DEV)
    else:
        s["codes"], s["scales"] = _to_block(randn(taken, kv, GROUP, d) * wide[:, None], randn(taken, kv, GROUP, d), c["fmt"])
    return s


def _prepare_attend(c, lens, visible, gen):
    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    B, kv, d = c["batch"], c["kv"], c["d"]
    shared = c["kind"] == "shared"
    s = {}
    s["slot_offset"], total = _offsets(lens, shared)
    s["block_offset"], blocks = _offsets([t // GROUP for t in lens], shared)
    blocks = max(blocks, 1)
    s["block_map"] = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    # complete groups live in the coded cache; the 32-bit cache is a small ring that holds the raw
    # tails (slots of coded tokens have been given back: slot 0)
    slots, at = torch.zeros(max(total, 1), dtype=torch.int32), 0
    for b, t in enumerate(lens):
        for i in range(t - t % GROUP, t):
            slots[at + i] = 1 + i % GROUP + (0 if shared else 3 * b)
        at += 0 if shared else t
    s["slot_map"] = slots.to(DEV)
    n = 4 + (0 if shared else 3 * B)
    s["k_cache"], s["v_cache"] = randn(n, kv, d), randn(n, kv, d)
    wide = 1 + 3 * (torch.rand(kv, 1, d, generator=gen, device=DEV) > 0.97)
    codes, scales = [], []
    for at in range(0, blocks, 1 << 16):
        m = min(1 << 16, blocks - at)
        # values of one block and the next differ in size
        size = 0.25 + 2 * torch.rand(m, 1, 1, 1, generator=gen, device=DEV)
        raw, sc = _to_block(randn(m, kv, GROUP, d) * wide, randn(m, kv, GROUP, d) * size, c["fmt"])
        codes.append(raw)
        scales.append(sc)
    s["codes"], s["scales"] = torch.cat(codes), torch.cat(scales)
    s["q"] = randn(B, c["heads"], d)
    if c["rows"]:
        s["ids"], s["n_ids"] = _rows(c, lens, visible, gen)
    if c["weights"]:
        s["weight_offset"], n = _offsets([-(-t // GROUP) for t in lens], shared)
        s["weights_before"] = 8 * torch.rand(max(n, 1), generator=gen, device=DEV)
        s["weights"] = s["weights_before"].clone()
    s["out"] = torch.zeros(B, c["heads"], d, device=DEV)
    return s


def _rows(c, lens, visible, gen):
    """Token rows as a selection emits them: ascending groups of four tokens, then the raw tail."""
    B, budget = c["batch"], c["rows"]
    gm = max(max(lens) // GROUP, 1)
    k = (visible // GROUP).clamp(max=budget).to(torch.int64)
    key = torch.rand(B, gm, generator=gen, device=DEV)
    key = key.masked_fill(torch.arange(gm, device=DEV)[None] >= (visible // GROUP)[:, None], 2.0)
    take = torch.topk(key, min(budget, gm), dim=1, largest=False).indices
    take = take.masked_fill(torch.arange(take.shape[1], device=DEV)[None] >= k[:, None], 1 << 40).sort(dim=1).values
    i = torch.arange(GROUP * budget + 3, device=DEV)[None].expand(B, -1)
    grp = torch.gather(take, 1, (i // GROUP).clamp(max=take.shape[1] - 1)) * GROUP + i % GROUP
    tail = visible[:, None] - visible[:, None] % GROUP + (i - GROUP * k[:, None])
    n = GROUP * k + visible % GROUP
    ids = torch.where(i < GROUP * k[:, None], grp, tail).masked_fill(i >= n[:, None], -1)
    return ids.to(torch.int32).contiguous(), n.to(torch.int32)


# ---- one pass ---------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _normed(x, w):
    x = x.to(torch.float32)
    return x if w is None else x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w


def _turned(x, cos, sin, pairing):
    """x [B, heads, width] with its first 2 * cos.shape[1] dims rotated, pair by pair."""
    half = cos.shape[1]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    cos, sin = cos[:, None], sin[:, None]
    if pairing == "halves":
        a, b = head[..., :half], head[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2), rest], dim=-1)


def _plain_append(s):
    c = s["case"]
    B = c["batch"]
    angles = {}
    for name in ("freq", "idx_freq"):
        a = (s["positions"].to(torch.float64)[:, :, None] * s[name].to(torch.float64)[:, None, :]).sum(dim=0)
        angles[name] = torch.cos(a).to(torch.float32), torch.sin(a).to(torch.float32)
    made = {}
    for name, width, freq in (("q", c["d"], "freq"), ("k", c["d"], "freq"), ("v", c["d"], None),
                              ("q_idx", c["idx"], "idx_freq"), ("idx_key", c["idx"], "idx_freq")):
        x = _normed(s["rows"][name].reshape(B, -1, width), s.get(name + "_norm"))
        made[name] = x if freq is None else _turned(x, *angles[freq], c["pairing"])
    has = s["visible"] > 0  # an empty history has no new token
    at = s["slot_offset"][has] + s["visible"][has] - 1
    slot = s["slot_map"][at].to(torch.int64)
    s["q"][has], s["q_idx"][has] = made["q"][has], made["q_idx"][has]
    s["k_cache"][slot], s["v_cache"][slot] = made["k"][has], made["v"][has]
    s["idx_keys"][at] = made["idx_key"][has, 0]
    return _appended(s)


def _appended(s):
    return {name: s[name] for name in ("q", "q_idx", "k_cache", "v_cache", "idx_keys")}


def _places(s):
    """Blocks and slots of the groups of a call."""
    g = s["group_begin"][:, None] + torch.arange(s["case"]["groups"], device=DEV)
    t = GROUP * g[..., None] + torch.arange(GROUP, device=DEV)
    return (s["block_map"][s["block_offset"][:, None] + g].to(torch.int64),
            s["slot_map"][s["slot_offset"][:, None, None] + t].to(torch.int64))


def _plain_read(s):
    c = s["case"]
    blk, slot = _places(s)
    k, v = _decoded(s["codes"][blk], s["scales"][blk], c["d"], c["fmt"])  # [B, groups, kv, 4, d]
    s["k_back"][slot], s["v_back"][slot] = k.transpose(2, 3), v.transpose(2, 3)
    return {"k": s["k_back"], "v": s["v_back"]}


def _plain_store(s):
    blk, slot = _places(s)
    raw, scales = _to_block(s["k_cache"][slot].transpose(2, 3), s["v_cache"][slot].transpose(2, 3), s["case"]["fmt"])
    s["codes"][blk], s["scales"][blk] = raw, scales
    return {**_plain_read(s), "scales": s["scales"]}


def _plain_attend(s):
    c = s["case"]
    B, nq, kv, d = c["batch"], c["heads"], c["kv"], c["d"]
    T = s["visible"].to(torch.int64)
    if c["rows"]:
        i = torch.arange(c["rows"], device=DEV)[None].expand(B, -1)
        ok = i < (s["n_ids"] // GROUP)[:, None]
        g = torch.where(ok, s["ids"][:, 0:GROUP * c["rows"]:GROUP] // GROUP, 0).to(torch.int64)
    else:
        g = torch.arange(max(c["tokens"] // GROUP, 1), device=DEV)[None].expand(B, -1)
        ok = g < (T // GROUP)[:, None]
        g = torch.where(ok, g, 0)
    n = g.shape[1]
    blk = s["block_map"][torch.where(ok, s["block_offset"][:, None] + g, 0)].to(torch.int64)
    K, V = _decoded(s["codes"][blk], s["scales"][blk], d, c["fmt"])  # [B, n, kv, 4, d]
    K, V = (x.transpose(1, 2).reshape(B, kv, n * GROUP, d) for x in (K, V))
    q = s["q"].reshape(B, kv, nq // kv, d)
    # the raw tail: the tokens behind the last complete group
    t = (T - T % GROUP)[:, None] + torch.arange(3, device=DEV)[None]
    in_tail = t < T[:, None]
    slot = s["slot_map"][torch.where(in_tail, s["slot_offset"][:, None] + t, 0)].to(torch.int64)
    Kt, Vt = s["k_cache"][slot].transpose(1, 2), s["v_cache"][slot].transpose(1, 2)  # [B, kv, 3, d]
    x = torch.cat([torch.matmul(q, K.transpose(2, 3)), torch.matmul(q, Kt.transpose(2, 3))], dim=3) * (1.0 / math.sqrt(d))
    seen = torch.cat([ok.repeat_interleave(GROUP, dim=1), in_tail], dim=1)[:, None, None, :]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(dim=3, keepdim=True)
    p = torch.where(seen, torch.exp(x - torch.where(m == -math.inf, 0.0, m)), 0.0)
    l = p.sum(dim=3, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    out = (torch.matmul(p[..., :n * GROUP], V) + torch.matmul(p[..., n * GROUP:], Vt)).reshape(B, nq, d)
    if not c["weights"]:
        return out
    mass = p.sum(dim=(1, 2), dtype=torch.float64)  # [B, tokens]: of every head
    per = torch.cat([mass[:, :n * GROUP].reshape(B, n, GROUP).sum(2), mass[:, n * GROUP:].sum(1, keepdim=True)], dim=1)
    at = s["weight_offset"][:, None] + torch.cat([g, (T // GROUP)[:, None]], dim=1)
    some = torch.cat([ok, (T % GROUP > 0)[:, None]], dim=1)
    w = s["weights_before"].to(torch.float64)
    w.index_add_(0, torch.where(some, at, 0).flatten(), torch.where(some, per, 0.0).flatten())
    return {"out": out, "weights": w.to(torch.float32)}


_plain = {"append": _plain_append, "store": _plain_store, "read": _plain_read, "attend": _plain_attend}


# ---- the library's calls ----------------------------------------------------------

def _plan(s):
    from top_group_sparse_gb300 import qsa
    c = s["case"]
    if c["op"] == "append":
        dims = qsa.make_dims(c["batch"], c["ih"], c["idx"], c["heads"], c["kv"], c["d"], max_visible=max(_lengths(c)))
        at = {k: s[k].data_ptr() for k in ("visible", "q", "q_idx", "idx_keys", "k_cache", "v_cache", "slot_map", "slot_offset")}
        pairing = qsa.QSA_PAIR_HALVES if c["pairing"] == "halves" else qsa.QSA_PAIR_NEIGHBOURS
        tokens = qsa.QsaNewTokens.of(**s["rows"], positions=s["positions"], freq=s["freq"], idx_freq=s["idx_freq"],
                                     pairing=pairing, eps=EPS,
                                     **{k: s[k] for k in ("q_norm", "k_norm", "q_idx_norm", "idx_key_norm")})
        return {"qsa": qsa, "dims": dims, "tokens": tokens,
                "inputs": qsa.QsaInputs(num_slots=s["k_cache"].shape[0], key_offset=at["slot_offset"], **at),
                "ws": torch.zeros(qsa.QSA_ROWS_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)}
    dims = qsa.make_dims(c["batch"], 8, 64, c.get("heads", c["kv"]), c["kv"], c["d"], budget_groups=c.get("rows") or 512,
                         max_visible=max(_lengths(c)))
    cache = qsa.QsaCodedCache.of(s["codes"], s["scales"], s["block_map"], s["block_offset"], FORMAT[c["fmt"]])
    at = {k: s[k].data_ptr() for k in ("visible", "slot_map", "slot_offset")}
    p = {"qsa": qsa, "dims": dims, "cache": cache}
    if c["op"] != "read":
        p["inputs"] = qsa.QsaInputs(k_cache=s["k_cache"].data_ptr(), v_cache=s["v_cache"].data_ptr(),
                                    num_slots=s["k_cache"].shape[0], q=s["q"].data_ptr() if "q" in s else None, **at)
    if c["op"] != "attend":
        p["back"] = qsa.QsaInputs(k_cache=s["k_back"].data_ptr(), v_cache=s["v_back"].data_ptr(),
                                  num_slots=s["k_back"].shape[0], **at)
    p["ws"] = torch.zeros(qsa.qsa_coded_workspace_size(dims, c["op"] == "attend" and not c["rows"], c.get("weights", False)),
                          dtype=torch.uint8, device=DEV)
    return p


def _own_append(s):
    p = s["plan"]
    p["qsa"].qsa_append_tokens(p["dims"], p["inputs"], p["tokens"], p["ws"])
    return _appended(s)


def _own_read(s):
    p = s["plan"]
    p["qsa"].qsa_read_groups(p["dims"], p["back"], p["cache"], s["group_begin"], s["group_end"], s["case"]["groups"], p["ws"])
    return {"k": s["k_back"], "v": s["v_back"]}


def _own_store(s):
    p = s["plan"]
    p["qsa"].qsa_code_groups(p["dims"], p["inputs"], p["cache"], s["group_begin"], s["group_end"], s["case"]["groups"],
                             p["ws"])
    return {**_own_read(s), "scales": s["scales"]}


def _own_attend(s):
    p = s["plan"]
    if not s["case"]["weights"]:
        p["qsa"].qsa_attend_coded(p["dims"], p["inputs"], p["cache"], s.get("ids"), s.get("n_ids"), s["out"], p["ws"])
        return s["out"]
    s["weights"].copy_(s["weights_before"])  # the accumulators as they were, so that a pass can be repeated
    p["qsa"].qsa_attend_coded(p["dims"], p["inputs"], p["cache"], s.get("ids"), s.get("n_ids"), s["out"], p["ws"],
                              weights=s["weights"], weight_offset=s["weight_offset"])
    return {"out": s["out"], "weights": s["weights"]}


_own = {"append": _own_append, "store": _own_store, "read": _own_read, "attend": _own_attend}


# ---- the definitions in 64 bits ------------------------------------------------------

def _e2m1(n):
    """The numbers that e2m1 codes stand for, from the format's definition."""
    e, m = (n >> 1) & 3, (n & 1).double()
    return torch.where(n >= 8, -1.0, 1.0) * torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))


def _e4m3(n):
    e, m = ((n >> 3) & 15).double(), (n & 7).double()
    return torch.where(n >= 128, -1.0, 1.0) * torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))


def _look(raw, fmt, d, token, dim):
    """(K, V) in 64 bits without the group's scale: the value at (token, dim) of blocks [..., bytes], by its place."""
    b = raw.to(torch.int32)
    if fmt in ("e4m3", "int8"):
        k = b[..., (dim // 64) * 256 + token * 64 + dim % 64]
        v = b[..., 4 * d + 4 * dim + token]
        return (_e4m3(k), _e4m3(v)) if fmt == "e4m3" else tuple(torch.where(x >= 128, x - 256, x).double() for x in (k, v))
    word = (dim // 64) * 128 + (token % 2) * 64 + (dim % 64 // 16) * 16 + (token // 2) * 8 + (dim % 16 // 8) * 4
    e = dim % 8
    nib = 2 * (e % 4) + e // 4 if fmt == "e2m1" else e
    k = (b[..., word + nib // 2] >> (4 * (nib % 2))) & 15
    word = 2 * d + (dim // 64) * 128 + (dim % 32 // 4) * 16 + (dim % 64 // 32) * 8 + (dim % 4 // 2) * 4
    p = 2 * (dim % 2) + token // 2
    nib = 2 * p + token % 2 if fmt == "e2m1" else p + 4 * (token % 2)
    v = (b[..., word + nib // 2] >> (4 * (nib % 2))) & 15
    kt = b[..., 4 * d + (dim % 64 // 16) * (d // 16) + 4 * (dim // 64) + dim % 16 // 4]
    vt = b[..., 4 * d + d // 4 + (dim % 32 // 4) * (d // 32) + dim // 32]
    k, v = (_e2m1(k), _e2m1(v)) if fmt == "e2m1" else (k.double() - 8, v.double() - 8)
    return k * _e4m3(kt), v * _e4m3(vt)


def _values(raw, scales, fmt, d):
    """K, V [n, 4, d] of blocks [n, bytes] with scales [n, 2]."""
    token, dim = torch.arange(GROUP, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    k, v = _look(raw, fmt, d, token, dim)
    return k * scales[:, 0].double()[:, None, None], v * scales[:, 1].double()[:, None, None]


def _nearest(x, bits, lowest):
    """x rounded to `bits` binary places after its leading one, ties to even; no step below 2^lowest."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60)))
    step = torch.exp2((e - bits).clamp(min=lowest))
    return torch.round(x / step) * step


def _stored(x, fmt):
    """(values, scales) in 64 bits that the coding of x [n, 4, d] stands for; products and quotients are binary32's."""
    top = TOP[fmt]
    x = x.double()
    scale = (x.abs().amax(dim=(1, 2)) * float(torch.tensor(1.0 / (448.0 * top), dtype=torch.float32))).float().double()
    scale = torch.where(scale >= 2.0 ** -126, scale, 0.0)
    most = x.abs().amax(dim=1).reshape(len(x), -1, 4).amax(dim=2)
    t = (most / (scale * top).float().double()[:, None]).float().double()
    t = torch.where(scale[:, None] > 0, _nearest(t, 3, -9).clamp(max=448.0), 0.0)
    s = (t * scale[:, None]).float().double().repeat_interleave(4, dim=1)[:, None]
    y = torch.where(s > 0, (x / s).float().double(), 0.0).clamp(-top, top)
    y = torch.round(y) if fmt == "int4" else _nearest(y, 1, -1)
    return y * (t * scale[:, None]).repeat_interleave(4, dim=1)[:, None], scale


def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "attend": _exact_attend}.get(c["op"], _exact_groups)(c, s)


def _exact_append(c, s):
    out = {k: v.double() for k, v in _appended(s).items()}
    lens = torch.tensor(_lengths(c), device=DEV)
    b = torch.nonzero(lens > 0)[:, 0]
    row = (s["slot_offset"] + lens - 1)[b]
    for name, width, freq in (("q", c["d"], "freq"), ("k", c["d"], "freq"), ("v", c["d"], None),
                              ("q_idx", c["idx"], "idx_freq"), ("idx_key", c["idx"], "idx_freq")):
        x = s["rows"][name][b].double().unflatten(1, (-1, width))
        w = s.get(name + "_norm")
        if w is not None:
            x = x / torch.sqrt(x.square().sum(dim=2, keepdim=True) / width + EPS) * w.double()
        if freq is not None and s[freq].shape[1]:
            half = s[freq].shape[1]
            angle = torch.einsum("ab,aj->bj", s["positions"][:, b].double(), s[freq].double())
            one, two = (slice(0, half), slice(half, 2 * half)) if c["pairing"] == "halves" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
            z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
            x[..., one], x[..., two] = z.real, z.imag
        if name in ("q", "q_idx"):
            out[name][b] = x
        elif name == "idx_key":
            out["idx_keys"][row] = x[:, 0]
        else:
            out[name + "_cache"][s["slot_map"][row].long()] = x
    return out


def _exact_groups(c, s):
    out = {"k": s["k_back"].double(), "v": s["v_back"].double()}
    if c["op"] == "store":
        out["scales"] = s["scales"].double()
    for b in range(c["batch"]):
        lo, hi = int(s["group_begin"][b]), int(s["group_end"][b])
        at, blk0 = int(s["slot_offset"][b]), int(s["block_offset"][b])
        slots = s["slot_map"][at + GROUP * lo:at + GROUP * hi].long()
        blk = s["block_map"][blk0 + lo:blk0 + hi].long()
        for h in range(c["kv"]):
            if c["op"] == "read":
                got = _values(s["codes"][blk, h], s["scales"][blk, h], c["fmt"], c["d"])
            else:
                got = []
                for i, cache in enumerate((s["k_cache"], s["v_cache"])):
                    x, out["scales"][blk, h, i] = _stored(cache[slots, h].unflatten(0, (hi - lo, GROUP)), c["fmt"])
                    got.append(x)
            out["k"][slots, h], out["v"][slots, h] = (x.flatten(0, 1) for x in got)
    return out


def _exact_attend(c, s):
    kv, d, nq = c["kv"], c["d"], c["heads"]
    out = torch.zeros(c["batch"], nq, d, dtype=torch.float64, device=DEV)
    w = s["weights_before"].double() if c["weights"] else None
    for b, t in enumerate(_lengths(c)):
        if t == 0:
            continue
        if c["rows"]:
            grp = s["ids"][b, :int(s["n_ids"][b]) - t % GROUP].long()[::GROUP] // GROUP
        else:
            grp = torch.arange(t // GROUP, device=DEV)
        blk = s["block_map"][int(s["block_offset"][b]) + grp].long()
        slots = s["slot_map"][int(s["slot_offset"][b]) + t - t % GROUP:int(s["slot_offset"][b]) + t].long()
        for h in range(kv):
            k, v = (x.reshape(-1, d) for x in _values(s["codes"][blk, h], s["scales"][blk, h], c["fmt"], d))
            k, v = torch.cat([k, s["k_cache"][slots, h].double()]), torch.cat([v, s["v_cache"][slots, h].double()])
            q = s["q"][b, h * (nq // kv):(h + 1) * (nq // kv)].double()
            p = torch.softmax(k @ q.T / math.sqrt(d), dim=0)  # [tokens, heads]
            out[b, h * (nq // kv):(h + 1) * (nq // kv)] = p.T @ v
            if w is not None:
                mass, first, n = p.sum(1), int(s["weight_offset"][b]), GROUP * len(grp)
                w[first + grp] += mass[:n].reshape(-1, GROUP).sum(1)
                if t % GROUP:
                    w[first + t // GROUP] += mass[n:].sum()
    return out if w is None else {"out": out, "weights": w}
