"""Cases of the 8-bit K/V cache and of the eviction that bounds a history.

Three operators, each with its plain form (elementary torch operations in 32
bits) and the library's call:

* ``code``   -- the K/V rows of complete four-token groups turned into 8-bit
  codes with one scale per (group, KV head) for K and one for V, and written
  into the blocks of the coded cache (``qsa_code_groups``);
* ``attend`` -- attention of one query per batch entry over the coded cache:
  over every visible token, or over the token rows that a selection emitted,
  with the attention weight that each group received added to running
  accumulators where the case asks for it (``qsa_attend_coded``);
* ``evict``  -- the groups a history keeps, by accumulated weight, and the
  history moved into its new place (``qsa_evict_select``,
  ``qsa_evict_compact``).

Codes are returned as numbers of their own 8-bit type (e4m3 or signed
integer) beside the scales that multiply them.
"""
import math
import random

import torch

own = False

GROUP = 4
DEV = "cuda"
QMAX = {"e4m3": 448.0, "int8": 127.0}
FORMAT = {"e4m3": 0, "int8": 1}


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # A decode step of 32 sequences in which every sequence completes a group: latency.
        dict(name="code_step", op="code", batch=32, tokens=2052, groups=1, kv=2, d=128, fmt="e4m3"),
        # A prompt's cache coded at once, after a chunked prefill of 100,000 positions.
        dict(name="code_prompt", op="code", batch=1, tokens=100255, groups=25063, kv=2, d=128, fmt="int8"),
        # The smallest history: one query, one head, 37 tokens (9 groups and one raw token).
        dict(name="attend_t37", op="attend", batch=1, tokens=37, kind="equal", rows=0, weights=False,
             heads=1, kv=1, d=64, fmt="e4m3"),
        # Layers that attend to everything: 8 long sequences.
        dict(name="attend_long", op="attend", batch=8, tokens=262144, kind="equal", rows=0, weights=False,
             heads=16, kv=2, d=128, fmt="e4m3"),
        # A serving batch of mixed lengths up to 65,537, an empty one and a raw tail alone among them.
        dict(name="attend_ragged", op="attend", batch=32, tokens=65537, kind="ragged", rows=0, weights=False,
             heads=16, kv=2, d=128, fmt="int8"),
        # Heads without sharing (one query head per KV head), head width 64.
        dict(name="attend_mha", op="attend", batch=12, tokens=9001, kind="ragged", rows=0, weights=False,
             heads=8, kv=8, d=64, fmt="int8"),
        # The observation pass before an eviction: every token's weight, sixteen query heads on one KV head.
        dict(name="attend_observe", op="attend", batch=4, tokens=40003, kind="equal", rows=0, weights=True,
             heads=16, kv=1, d=128, fmt="int8"),
        # Decode over selected rows: 512 groups of each of 8 long histories.
        dict(name="rows_long", op="attend", batch=8, tokens=262144, kind="equal", rows=512, weights=False,
             heads=16, kv=2, d=128, fmt="e4m3"),
        # A chunk of 256 consecutive positions of one history, each with its own selected rows; what
        # they attend to is accumulated for the history that they share.
        dict(name="rows_chunk", op="attend", batch=256, tokens=100256, kind="shared", rows=512, weights=True,
             heads=16, kv=2, d=128, fmt="e4m3"),
        # Three short histories cut to 512 groups: latency.
        dict(name="evict_short", op="evict", batch=3, tokens=4099, kind="ragged", keep=512, sink=1, recent=16,
             idx=32),
        # Eight long histories cut to half.
        dict(name="evict_long", op="evict", batch=8, tokens=262144, kind="equal", keep=32768, sink=4, recent=64,
             idx=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["code", "attend", "attend", "attend", "evict"])
    fmt = rng.choice(["e4m3", "int8"])
    heads, kv, d = rng.choice([(1, 1, 64), (2, 2, 64), (8, 8, 64), (8, 2, 64), (16, 2, 128), (16, 1, 128),
                               (32, 8, 128), (12, 4, 128), (10, 2, 128)])
    if op == "code":
        batch = _log(rng, 1, 64)
        groups = _log(rng, 1, 2 ** 17 // (batch * kv))
        tokens = GROUP * (groups + rng.randrange(0, 500)) + rng.randrange(4)
        return dict(op=op, batch=batch, tokens=tokens, groups=groups, kv=kv, d=d, fmt=fmt)
    if op == "evict":
        batch = _log(rng, 1, 8)
        tokens = _log(rng, 64, 262144)
        groups = tokens // GROUP
        keep = max(2, int(groups * rng.uniform(0.2, 0.75)))
        sink = rng.randrange(0, min(9, keep // 2 + 1))
        recent = rng.randrange(0, min(65, keep - sink + 1))
        return dict(op=op, batch=batch, tokens=tokens, kind=rng.choice(["equal", "ragged"]), keep=keep, sink=sink,
                    recent=recent, idx=rng.choice([32, 64]))
    most = 2 ** 30 // (2 * kv * d)  # tokens in all
    kind = rng.choice(["equal", "ragged", "ragged", "shared"])
    rows = rng.choice([0, 0, 512, _log(rng, 1, 512)])
    if rows:
        batch = _log(rng, 1, 256 if kind == "shared" else 32)
        tokens = _log(rng, 1, min(262144, most // (1 if kind == "shared" else batch)))
    else:  # every query reads its whole history
        batch = _log(rng, 1, 32)
        tokens = _log(rng, 1, min(262144, most // batch))
    return dict(op=op, batch=batch, tokens=max(tokens, batch if kind == "shared" else 1), kind=kind, rows=rows,
                weights=rng.random() < 0.4, heads=heads, kv=kv, d=d, fmt=fmt)


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


def work(c):
    if c["op"] == "code":
        n = c["batch"] * c["groups"] * c["kv"] * 2  # K and V of one block and head
        return {"bytes": n * (GROUP * c["d"] * 5 + 4) + c["batch"] * c["groups"] * 20, "flops": n * GROUP * c["d"] * 2}
    lens = _lengths(c)
    if c["op"] == "evict":
        kept = sum(min(t // GROUP, c["keep"]) for t in lens)
        tail = sum(t % GROUP for t in lens)
        per = 2 * (5 * c["idx"] * 4 + 4 * 4 + 4 + 4) + 4
        return {"bytes": sum(t // GROUP for t in lens) * 4 + kept * per + tail * 2 * (c["idx"] * 4 + 4), "flops": 0}
    kv, d, nq = c["kv"], c["d"], c["heads"]
    groups = [min(t // GROUP, c["rows"]) if c["rows"] else t // GROUP for t in lens]
    # queries of one history share what they read
    blocks = sum(groups) if c["kind"] != "shared" else min(sum(groups), max(lens) // GROUP)
    tail = sum(t % GROUP for t in lens)
    per = kv * (8 * d + 8) + 4
    moved = blocks * per + tail * kv * d * 8 + len(lens) * nq * d * 8
    if c["rows"]:
        moved += sum(groups) * 16
    if c["weights"]:
        moved += blocks * 8
    return {"bytes": moved, "flops": 4 * nq * d * sum(GROUP * g + t % GROUP for g, t in zip(groups, lens))}


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


def _to_codes(x, fmt):
    """8-bit codes (as bytes) and scales of x [..., 4, d] over its last two axes."""
    amax = x.abs().amax(dim=(-2, -1))
    scale = amax / QMAX[fmt]
    scale = torch.where(scale >= 2.0 ** -126, scale, torch.zeros_like(scale))
    y = x / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None, None]
    y = torch.where((scale > 0)[..., None, None], y, torch.zeros_like(y)).clamp(-QMAX[fmt], QMAX[fmt])
    code = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(y).to(torch.int8)
    return code.view(torch.uint8), scale


def _pack(kc, vc):
    """Codes of K and V [..., 4, d] in a block's layout: K as [d/64][4][64], V as [d][4]."""
    d = kc.shape[-1]
    k = kc.unflatten(-1, (d // 64, 64)).transpose(-3, -2).flatten(-3)
    v = vc.transpose(-1, -2).flatten(-2)
    return torch.cat([k, v], dim=-1)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    lens = _lengths(c)
    B = c["batch"]
    shared = c.get("kind") == "shared"
    s = {"case": c, "visible": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if c["op"] == "evict":
        s |= _prepare_evict(c, lens, gen)
    else:
        kv, d = c["kv"], c["d"]
        s["slot_offset"], total = _offsets(lens, shared)
        s["block_offset"], blocks = _offsets([t // GROUP for t in lens], shared)
        blocks = max(blocks, 1)
        s["block_map"] = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
        if c["op"] == "code":
            # the raw rows still sit in the 32-bit cache, in pages of 16 tokens; a sequence's last
            # `groups` groups are coded by the call
            pages = -(-max(total, 1) // 16)
            perm = torch.randperm(pages, generator=gen, device=DEV)
            t = torch.arange(max(total, 1), device=DEV)
            s["slot_map"] = (perm[t // 16] * 16 + t % 16).to(torch.int32)
            # keys carry a few wide channels, as trained projections do
            wide = 1 + 7 * (torch.rand(kv, d, generator=gen, device=DEV) > 0.95)
            s["k_cache"] = randn(pages * 16, kv, d) * wide
            s["v_cache"] = randn(pages * 16, kv, d)
            s["codes"] = torch.zeros(blocks, kv, 8 * d, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros(blocks, kv, 2, device=DEV)
            end = s["visible"] // GROUP
            s["group_begin"], s["group_end"] = (end - c["groups"]).contiguous(), end.contiguous()
        else:
            # complete groups live in the coded cache; the 32-bit cache is a small ring that holds the
            # raw tails (slots of coded tokens have been given back: slot 0)
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
                kc, ks = _to_codes(randn(m, kv, GROUP, d) * wide, c["fmt"])
                # values of one block and the next differ in size
                vc, vs = _to_codes(randn(m, kv, GROUP, d) * (0.25 + 2 * torch.rand(m, 1, 1, 1, generator=gen,
                                                                                   device=DEV)), c["fmt"])
                codes.append(_pack(kc, vc))
                scales.append(torch.stack([ks, vs], dim=-1))
            s["codes"], s["scales"] = torch.cat(codes), torch.cat(scales)
            s["q"] = randn(B, c["heads"], d)
            if c["rows"]:
                s["ids"], s["n_ids"] = _rows(c, lens, s["visible"], gen)
            if c["weights"]:
                s["weight_offset"], n = _offsets([-(-t // GROUP) for t in lens], shared)
                s["weights_before"] = 8 * torch.rand(max(n, 1), generator=gen, device=DEV)
                s["weights"] = s["weights_before"].clone()
            s["out"] = torch.zeros(B, c["heads"], d, device=DEV)
    if own:
        s["plan"] = _plan(s)
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


def _prepare_evict(c, lens, gen):
    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    idx = c["idx"]
    groups = [t // GROUP for t in lens]
    kept = [min(g, c["keep"]) for g in groups]
    after = [GROUP * k + t % GROUP for k, t in zip(kept, lens)]
    s = {}
    for side, ts in (("src", lens), ("dst", after)):
        tok, nt = _offsets(ts)
        grp, ng = _offsets([t // GROUP for t in ts])
        wgt, nw = _offsets([-(-t // GROUP) for t in ts])
        nt, ng, nw = max(nt, 1), max(ng, 1), max(nw, 1)
        if side == "src":
            # most groups of a long history got next to nothing, many nothing at all: ties
            w = torch.exp(2.5 * randn(nw)) * (torch.rand(nw, generator=gen, device=DEV) > 0.5)
            h = {"idx_keys": randn(nt, idx), "pooled": randn(ng, idx), "weights": w,
                 "slot_map": torch.randperm(nt, generator=gen, device=DEV).to(torch.int32),
                 "block_map": torch.randperm(ng, generator=gen, device=DEV).to(torch.int32),
                 "visible": torch.tensor(ts, dtype=torch.int32, device=DEV)}
        else:
            h = {"idx_keys": torch.zeros(nt, idx, device=DEV), "pooled": torch.zeros(ng, idx, device=DEV),
                 "weights": torch.zeros(nw, device=DEV),
                 "slot_map": torch.zeros(nt, dtype=torch.int32, device=DEV),
                 "block_map": torch.zeros(ng, dtype=torch.int32, device=DEV),
                 "visible": torch.zeros(len(ts), dtype=torch.int32, device=DEV)}
        h |= {"key_offset": tok, "slot_offset": tok, "pool_offset": grp, "block_offset": grp, "weight_offset": wgt}
        s[side] = h
    s["kept"] = torch.full((len(lens), c["keep"]), -1, dtype=torch.int32, device=DEV)
    s["n_kept"] = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _plain_code(s):
    c = s["case"]
    j = torch.arange(c["groups"], device=DEV)
    g = s["group_begin"][:, None] + j[None]
    t = GROUP * g[..., None] + torch.arange(GROUP, device=DEV)
    slot = s["slot_map"][s["slot_offset"][:, None, None] + t].to(torch.int64)
    kc, ks = _to_codes(s["k_cache"][slot].transpose(2, 3), c["fmt"])  # [B, groups, kv, 4, d]
    vc, vs = _to_codes(s["v_cache"][slot].transpose(2, 3), c["fmt"])
    blk = s["block_map"][s["block_offset"][:, None] + g].to(torch.int64)
    s["codes"][blk] = _pack(kc, vc)
    s["scales"][blk] = torch.stack([ks, vs], dim=-1)
    return _coded(s)


def _coded(s):
    """The codes as numbers of their own type, and the scales that multiply them."""
    kind = torch.float8_e4m3fn if s["case"]["fmt"] == "e4m3" else torch.int8
    return {"codes": s["codes"].view(kind), "scales": s["scales"]}


def _plain_attend(s):
    c = s["case"]
    B, nq, kv, d = c["batch"], c["heads"], c["kv"], c["d"]
    r = nq // kv
    T = s["visible"].to(torch.int64)
    scale = 1.0 / math.sqrt(d)
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
    kind = torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.int8
    raw, sc = s["codes"][blk], s["scales"][blk].permute(0, 2, 1, 3)  # [B, n, kv, 8d], [B, kv, n, 2]
    K = raw[..., :4 * d].reshape(B, n, kv, d // 64, GROUP, 64).permute(0, 2, 1, 4, 3, 5).contiguous()
    K = (K.view(kind).to(torch.float32).reshape(B, kv, n, GROUP * d) * sc[..., 0:1]).reshape(B, kv, n * GROUP, d)
    V = raw[..., 4 * d:].reshape(B, n, kv, d, GROUP).permute(0, 2, 1, 4, 3).contiguous()
    V = (V.view(kind).to(torch.float32).reshape(B, kv, n, GROUP * d) * sc[..., 1:2]).reshape(B, kv, n * GROUP, d)
    q = s["q"].reshape(B, kv, r, d)
    # the raw tail: the tokens behind the last complete group
    t = (T - T % GROUP)[:, None] + torch.arange(3, device=DEV)[None]
    in_tail = t < T[:, None]
    slot = s["slot_map"][torch.where(in_tail, s["slot_offset"][:, None] + t, 0)].to(torch.int64)
    Kt, Vt = s["k_cache"][slot].transpose(1, 2), s["v_cache"][slot].transpose(1, 2)  # [B, kv, 3, d]
    x = torch.cat([torch.matmul(q, K.transpose(2, 3)), torch.matmul(q, Kt.transpose(2, 3))], dim=3) * scale
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


def _plain_evict(s):
    c, src, dst = s["case"], s["src"], s["dst"]
    B, keep = c["batch"], c["keep"]
    T = src["visible"].to(torch.int64)
    G = T // GROUP
    gm = max(c["tokens"] // GROUP, 1)
    g = torch.arange(gm, device=DEV)[None].expand(B, -1)
    ok = g < G[:, None]
    w = torch.where(ok, src["weights"][torch.where(ok, src["weight_offset"][:, None] + g, 0)], -math.inf)
    w = torch.where(ok & ((g < c["sink"]) | (g >= G[:, None] - c["recent"])), math.inf, w)
    order = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :keep]
    n = G.clamp(max=keep)
    i = torch.arange(order.shape[1], device=DEV)[None]
    kept = torch.where(i < n[:, None], order, 1 << 40).sort(dim=1).values
    have = i < n[:, None]
    s["kept"][:, :kept.shape[1]] = torch.where(have, kept, -1).to(torch.int32)
    s["n_kept"].copy_(n)
    kept = torch.where(have, kept, 0)
    # whole groups; what is behind a row's end is written again with the row's first entry
    some = (n > 0)[:, None]
    i = torch.where(have, i, 0)
    kept = torch.where(have, kept, kept[:, :1])
    a, b = (src["pool_offset"][:, None] + kept)[some.expand_as(i)], (dst["pool_offset"][:, None] + i)[some.expand_as(i)]
    k8, i8 = (kept & 7)[some.expand_as(i)], (i & 7).expand(B, -1)[some.expand_as(i)]
    idx = c["idx"]
    chunk = torch.arange(idx // 4, device=DEV)[None] ^ (k8 ^ i8)[:, None]
    rows = torch.gather(src["pooled"][a].reshape(-1, idx // 4, 4), 1, chunk[..., None].expand(-1, -1, 4))
    dst["pooled"][b] = rows.reshape(-1, idx)
    dst["block_map"][b] = src["block_map"][a]
    wa, wb = src["weight_offset"][:, None] + kept, dst["weight_offset"][:, None] + i
    dst["weights"][wb[some.expand_as(i)]] = src["weights"][wa[some.expand_as(i)]]
    u = torch.arange(GROUP, device=DEV)
    ta = (src["key_offset"][:, None, None] + GROUP * kept[..., None] + u)[some.expand_as(i)]
    tb = (dst["key_offset"][:, None, None] + GROUP * i[..., None] + u)[some.expand_as(i)]
    dst["idx_keys"][tb] = src["idx_keys"][ta]
    dst["slot_map"][tb] = src["slot_map"][ta]
    # the raw tail
    j = torch.arange(3, device=DEV)[None].expand(B, -1)
    tail = j < (T % GROUP)[:, None]
    ta, tb = (src["key_offset"] + GROUP * G)[:, None] + j, (dst["key_offset"] + GROUP * n)[:, None] + j
    dst["idx_keys"][tb[tail]] = src["idx_keys"][ta[tail]]
    dst["slot_map"][tb[tail]] = src["slot_map"][ta[tail]]
    part = T % GROUP > 0
    dst["weights"][(dst["weight_offset"] + n)[part]] = src["weights"][(src["weight_offset"] + G)[part]]
    dst["visible"].copy_(GROUP * n + T % GROUP)
    return _evicted(s)


def _evicted(s):
    names = ("idx_keys", "pooled", "slot_map", "block_map", "weights", "visible")
    return {"kept": s["kept"], "n_kept": s["n_kept"], **{k: s["dst"][k] for k in names}}


_plain = {"code": _plain_code, "attend": _plain_attend, "evict": _plain_evict}


# ---- the library's calls ----------------------------------------------------------

def _plan(s):
    from top_group_sparse_gb300 import qsa
    c = s["case"]
    if c["op"] == "evict":
        dims = qsa.make_dims(c["batch"], 8, c["idx"], 16, 2, 128, max_visible=max(_lengths(c)))
        ws = torch.zeros(qsa.qsa_workspace_size(dims), dtype=torch.uint8, device=DEV)
        return {"qsa": qsa, "dims": dims, "ws": ws, "src": qsa.QsaHistory.of(**s["src"]),
                "dst": qsa.QsaHistory.of(**s["dst"])}
    dims = qsa.make_dims(c["batch"], 8, 64, c.get("heads", c["kv"]), c["kv"], c["d"], budget_groups=c.get("rows") or 512,
                         max_visible=max(_lengths(c)))
    ws = torch.zeros(qsa.qsa_coded_workspace_size(dims, c["op"] == "attend" and not c["rows"],
                                                  c.get("weights", False)), dtype=torch.uint8, device=DEV)
    at = {k: s[k].data_ptr() for k in ("visible", "k_cache", "v_cache", "slot_map", "slot_offset")}
    inp = qsa.QsaInputs(q=s["q"].data_ptr() if "q" in s else None, num_slots=s["k_cache"].shape[0], **at)
    cache = qsa.QsaCodedCache.of(s["codes"], s["scales"], s["block_map"], s["block_offset"], FORMAT[c["fmt"]])
    return {"qsa": qsa, "dims": dims, "ws": ws, "inputs": inp, "cache": cache}


def _own_code(s):
    p = s["plan"]
    p["qsa"].qsa_code_groups(p["dims"], p["inputs"], p["cache"], s["group_begin"], s["group_end"], s["case"]["groups"],
                             p["ws"])
    return _coded(s)


def _own_attend(s):
    p = s["plan"]
    if not s["case"]["weights"]:
        p["qsa"].qsa_attend_coded(p["dims"], p["inputs"], p["cache"], s.get("ids"), s.get("n_ids"), s["out"], p["ws"])
        return s["out"]
    s["weights"].copy_(s["weights_before"])  # the accumulators as they were, so that a pass can be repeated
    p["qsa"].qsa_attend_coded(p["dims"], p["inputs"], p["cache"], s.get("ids"), s.get("n_ids"), s["out"], p["ws"],
                              weights=s["weights"], weight_offset=s["weight_offset"])
    return {"out": s["out"], "weights": s["weights"]}


def _own_evict(s):
    p, c = s["plan"], s["case"]
    p["qsa"].qsa_evict_select(p["dims"], s["src"]["visible"], s["src"]["weights"], s["src"]["weight_offset"], c["keep"],
                              c["sink"], c["recent"], s["kept"], s["n_kept"], p["ws"])
    p["qsa"].qsa_evict_compact(p["dims"], c["keep"], s["kept"], s["n_kept"], p["src"], p["dst"], p["ws"])
    return _evicted(s)


_own = {"code": _own_code, "attend": _own_attend, "evict": _own_evict}


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "evict":
        return None  # copies and whole numbers
    if c["op"] == "code":
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV)
        for b in range(c["batch"]):
            lo, hi = int(s["group_begin"][b]), int(s["group_end"][b])
            at, blk0 = int(s["slot_offset"][b]), int(s["block_offset"][b])
            slots = s["slot_map"][at + GROUP * lo:at + GROUP * hi].long()
            blk = s["block_map"][blk0 + lo:blk0 + hi].long()
            for i, cache in enumerate((s["k_cache"], s["v_cache"])):
                rows = cache[slots].double().unflatten(0, (hi - lo, GROUP))
                scales[blk, :, i] = rows.abs().amax(dim=(1, 3)) / QMAX[c["fmt"]]
        return {"codes": None, "scales": scales}
    kv, d, nq = c["kv"], c["d"], c["heads"]
    kind = torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.int8
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
            codes = s["codes"][blk, h].view(kind).double()
            k = torch.cat([codes[:, 64 * GROUP * j:64 * GROUP * (j + 1)].reshape(-1, GROUP, 64) for j in range(d // 64)], 2)
            v = codes[:, GROUP * d:].reshape(-1, d, GROUP).mT
            k = (k * s["scales"][blk, h, 0].double()[:, None, None]).reshape(-1, d)
            v = (v * s["scales"][blk, h, 1].double()[:, None, None]).reshape(-1, d)
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
