"""Eviction by accumulated weight on the GPU against its definition
(tests/cache_helpers.py), and the operators of the bounded cache run together."""
import numpy as np
import pytest

import cache_helpers as ch
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


def _select(visible, weights, offset, keep, sink, recent, max_visible=None, with_evicted=True):
    import torch
    from top_group_sparse_gb300 import qsa
    B = len(visible)
    mv = int(max(visible)) if max_visible is None else max_visible
    dims = qsa.make_dims(B, 8, 64, 16, 2, 128, max_visible=mv)
    ws = torch.zeros(qsa.qsa_workspace_size(dims), dtype=torch.uint8, device="cuda")
    kept = torch.full((B, keep), -5, dtype=torch.int32, device="cuda")
    n_kept = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    ev = torch.full((B, max(mv // 4, 1)), -5, dtype=torch.int32, device="cuda") if with_evicted else None
    vis = torch.tensor(list(visible), dtype=torch.int32, device="cuda")
    qsa.qsa_evict_select(dims, vis, torch.as_tensor(weights).cuda(), torch.as_tensor(offset).cuda(), keep, sink, recent, kept,
                         n_kept, ws, evicted=ev)
    st, flags = qsa.qsa_check_errors(ws)
    return kept.cpu().numpy(), n_kept.cpu().numpy(), None if ev is None else ev.cpu().numpy(), flags


def _check(visible, weights, offset, keep, sink, recent, **kw):
    kept, n, ev, flags = _select(visible, weights, offset, keep, sink, recent, **kw)
    assert flags == 0
    want = ch.evict(visible, weights, offset, keep, sink, recent)
    for b, T in enumerate(visible):
        k = want[b]
        assert n[b] == len(k)
        assert np.array_equal(kept[b, :len(k)], k), f"query {b}"
        assert (kept[b, len(k):] == -5).all()
        if ev is not None:
            rest = np.setdiff1d(np.arange(int(T) // 4), k)
            assert np.array_equal(ev[b, :len(rest)], rest)
            assert (ev[b, len(rest):] == -5).all()


def _weights(n, kind, seed):
    r = np.random.RandomState(seed)
    w = np.exp(2.5 * r.randn(n)).astype(np.float32)
    if kind == "zeros":      # most groups got nothing
        w[r.rand(n) < 0.9] = 0
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "few":      # a handful of values
        w = r.randint(-2, 3, n).astype(np.float32)
        w[r.rand(n) < 0.1] = -0.0
    elif kind == "odd":      # infinities, NaN, subnormals, neighbours that differ in the last bit
        w = (np.float32(1.0).view(np.uint32) + r.randint(0, 4, n).astype(np.uint32)).astype(np.uint32).view(np.float32)
        for v in (np.inf, -np.inf, np.nan, 1e-44, -1e-44, 3.4e38):
            w[r.rand(n) < 0.05] = v
    return w


@pytest.mark.parametrize("kind", ["spread", "zeros", "equal", "few", "odd"])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 2, 3), (100, 0, 0), (100, 60, 40), (512, 4, 64),
                                              (1023, 1, 1)])
def test_the_kept_groups_equal_the_definition(kind, keep, sink, recent):
    need_gpu()
    visible = [0, 3, 4, 5, 28, 29, 400, 404, 407, 2052, 4096, 4099, 4 * 4095 + 2]
    offset = np.concatenate([[0], np.cumsum([-(-t // 4) for t in visible])])[:-1].astype(np.int64)
    w = _weights(int(offset[-1]) + 4096, kind, keep)
    _check(visible, w, offset, keep, sink, recent)


@pytest.mark.parametrize("kind", ["spread", "zeros", "odd"])
def test_long_histories_are_split_over_a_cluster(kind):
    need_gpu()
    for visible, keep in (([4 * 4097, 4 * 8191 + 3, 40000, 16388], 3000), ([262144, 262143, 100000], 32768), ([262144], 65535),
                          ([262144], 1)):
        offset = np.concatenate([[0], np.cumsum([-(-t // 4) for t in visible])])[:-1].astype(np.int64)
        w = _weights(int(offset[-1]) + 65536, kind, 7)
        _check(visible, w, offset, keep, min(4, keep), 0 if keep == 1 else 64, with_evicted=keep != 1)


def test_slices_longer_than_shared_memory_are_read_again():
    """More than 8 x 40,960 groups: the slices stay in device memory."""
    need_gpu()
    visible = [4 * 400001 + 1, 4 * 50]
    offset = np.array([5, 5 + 400002], np.int64)
    w = _weights(5 + 400002 + 51, "zeros", 9)
    _check(visible, w, offset, 150000, 4, 64)
    _check(visible[:1], w, offset[:1], 2, 0, 0, max_visible=1 << 26, with_evicted=False)


def test_a_length_out_of_range_keeps_nothing():
    need_gpu()
    from top_group_sparse_gb300 import qsa
    w = np.arange(100, dtype=np.float32)
    kept, n, ev, flags = _select([40, -4, 41], w, np.array([0, 20, 40]), 5, 0, 0, max_visible=40)
    assert flags == qsa.QSA_DEVERR_VISIBLE_RANGE
    assert n.tolist() == [5, 0, 0] and (kept[1:] == -5).all() and (ev[1:] == -5).all()
    assert kept[0].tolist() == [5, 6, 7, 8, 9]


# ---- the move ------------------------------------------------------------------------

def _history(visible, idx_dim, seed, fill=None):
    """Host arrays of histories with gaps between their regions."""
    r = np.random.RandomState(seed)

    def off(sizes):
        return np.concatenate([[3], 3 + np.cumsum([s + 5 for s in sizes])]).astype(np.int64)

    tok, grp, wgt = off(visible), off([t // 4 for t in visible]), off([-(-t // 4) for t in visible])
    h = {"idx_keys": r.randn(int(tok[-1]), idx_dim).astype(np.float32), "key_offset": tok[:-1],
         "pooled": r.randn(int(grp[-1]), idx_dim).astype(np.float32), "pool_offset": grp[:-1],
         "slot_map": r.randint(0, 1 << 30, int(tok[-1])).astype(np.int32), "slot_offset": tok[:-1],
         "block_map": r.randint(0, 1 << 30, int(grp[-1])).astype(np.int32), "block_offset": grp[:-1],
         "weights": r.rand(int(wgt[-1])).astype(np.float32), "weight_offset": wgt[:-1],
         "visible": np.asarray(visible, np.int32)}
    if fill is not None:
        for k in ("idx_keys", "pooled", "slot_map", "block_map", "weights", "visible"):
            h[k] = np.full_like(h[k], fill)
    return h


def _swizzled(rows, pos):
    """Pooled rows in the layout of their position: 16-byte chunk c at c ^ (pos & 7)."""
    out = np.empty_like(rows).reshape(len(rows), rows.shape[1] // 4, 4)
    for i, p in enumerate(pos):
        for c in range(out.shape[1]):
            out[i, c ^ (p & 7)] = rows[i].reshape(-1, 4)[c]
    return out.reshape(rows.shape)


def _moved(src, dst, kept, idx_dim):
    """dst as it is after the move, from the definition."""
    want = {k: v.copy() for k, v in dst.items()}
    for b, T in enumerate(src["visible"]):
        T, k = int(T), np.asarray(kept[b], np.int64)
        n, G = len(k), T // 4
        tok = np.concatenate([(4 * k[:, None] + np.arange(4)).ravel(), np.arange(4 * G, T)]).astype(np.int64)
        for a, o in (("idx_keys", "key_offset"), ("slot_map", "slot_offset")):
            want[a][dst[o][b]:dst[o][b] + len(tok)] = src[a][src[o][b] + tok]
        want["block_map"][dst["block_offset"][b]:dst["block_offset"][b] + n] = src["block_map"][src["block_offset"][b] + k]
        wk = np.concatenate([k, [G]]) if T % 4 else k
        want["weights"][dst["weight_offset"][b]:dst["weight_offset"][b] + len(wk)] = src["weights"][src["weight_offset"][b] + wk]
        rows = src["pooled"][src["pool_offset"][b] + k]
        plain = _swizzled(rows, k)  # the swizzle is its own inverse
        want["pooled"][dst["pool_offset"][b]:dst["pool_offset"][b] + n] = _swizzled(plain, np.arange(n))
        want["visible"][b] = 4 * n + T % 4
    return want


@pytest.mark.parametrize("idx_dim", [32, 64])
@pytest.mark.parametrize("keep", [1, 9, 100, 700])
def test_the_move_equals_the_definition(idx_dim, keep):
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    visible = [0, 1, 3, 4, 39, 40, 402, 2051, 2803]
    src = _history(visible, idx_dim, 1)
    kept = ch.evict(visible, src["weights"], src["weight_offset"], keep, 0, min(2, keep))
    dst = _history([4 * len(k) + t % 4 for k, t in zip(kept, visible)], idx_dim, 2, fill=-7)
    want = _moved(src, dst, kept, idx_dim)
    dims = qsa.make_dims(len(visible), 8, idx_dim, 16, 2, 128, max_visible=max(visible))
    ws = torch.zeros(qsa.qsa_workspace_size(dims), dtype=torch.uint8, device="cuda")
    kt = np.full((len(visible), keep), -9, np.int32)
    for b, k in enumerate(kept):
        kt[b, :len(k)] = k
    kt, nt = torch.from_numpy(kt).cuda(), torch.tensor([len(k) for k in kept], dtype=torch.int32, device="cuda")
    s = {k: torch.from_numpy(v).cuda() for k, v in src.items()}
    for left_out in ((), ("pooled",), ("idx_keys", "weights"), ("slot_map", "block_map")):
        d = {k: torch.from_numpy(v.copy()).cuda() for k, v in dst.items()}
        names = [k for k in s if k not in left_out]
        qsa.qsa_evict_compact(dims, keep, kt, nt, qsa.QsaHistory.of(**{k: s[k] for k in names}),
                              qsa.QsaHistory.of(**{k: d[k] for k in names}), ws)
        st, flags = qsa.qsa_check_errors(ws)
        assert flags == 0
        for k in d:
            ref = dst[k] if k in left_out else want[k]
            assert np.array_equal(d[k].cpu().numpy(), ref), (k, left_out)


def test_a_captured_eviction_replays_on_new_weights():
    """Selection and move captured once; replayed, they go by the weights of the day."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    visible, keep = [403, 40000], 50
    src = _history(visible, 64, 5)
    dims = qsa.make_dims(2, 8, 64, 16, 2, 128, max_visible=max(visible))
    ws = torch.zeros(qsa.qsa_workspace_size(dims), dtype=torch.uint8, device="cuda")
    dst = _history([4 * keep + t % 4 for t in visible], 64, 6, fill=-7)
    s = {k: torch.from_numpy(v).cuda() for k, v in src.items()}
    d = {k: torch.from_numpy(v.copy()).cuda() for k, v in dst.items()}
    kept = torch.full((2, keep), -1, dtype=torch.int32, device="cuda")
    n_kept = torch.zeros(2, dtype=torch.int32, device="cuda")

    def run():
        qsa.qsa_evict_select(dims, s["visible"], s["weights"], s["weight_offset"], keep, 1, 3, kept, n_kept, ws)
        qsa.qsa_evict_compact(dims, keep, kept, n_kept, qsa.QsaHistory.of(**s), qsa.QsaHistory.of(**d), ws)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (7, 8):
        src["weights"] = np.random.RandomState(seed).rand(len(src["weights"])).astype(np.float32)
        s["weights"].copy_(torch.from_numpy(src["weights"]))
        g.replay()
        assert qsa.qsa_check_errors(ws)[1] == 0
        want = ch.evict(visible, src["weights"], src["weight_offset"], keep, 1, 3)
        assert np.array_equal(kept.cpu().numpy(), np.array(want))
        moved = _moved(src, dst, want, 64)
        for k in d:
            assert np.array_equal(d[k].cpu().numpy(), moved[k]), k


def test_the_move_flags_what_is_out_of_range():
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    visible = [40, 41, 43, 48]
    src, dst = _history(visible, 64, 3), _history(visible, 64, 4, fill=-7)
    dims = qsa.make_dims(4, 8, 64, 16, 2, 128, max_visible=48)
    ws = torch.zeros(qsa.qsa_workspace_size(dims), dtype=torch.uint8, device="cuda")
    s = {k: torch.from_numpy(v).cuda() for k, v in src.items()}
    kept = torch.arange(6, dtype=torch.int32, device="cuda").repeat(4, 1)
    for n, vis, flag in (([6, -1, 7, 3], visible, qsa.QSA_DEVERR_ROW_RANGE), ([6, 2, 2, 2], [40, -1, 49, 48], qsa.QSA_DEVERR_VISIBLE_RANGE)):
        d = {k: torch.from_numpy(v.copy()).cuda() for k, v in dst.items()}
        s["visible"].copy_(torch.tensor(vis, dtype=torch.int32))
        qsa.qsa_evict_compact(dims, 6, kept, torch.tensor(n, dtype=torch.int32, device="cuda"), qsa.QsaHistory.of(**s),
                              qsa.QsaHistory.of(**d), ws)
        assert qsa.qsa_check_errors(ws)[1] == flag
        assert d["visible"].tolist() == [24, 0, 0, 4 * n[3]]
        for b in (1, 2):  # left out
            lo = int(dst["key_offset"][b])
            assert (d["idx_keys"][lo:lo + 20] == -7).all()
    # a position outside the history: zero rows, entries of -1
    s["visible"].copy_(torch.tensor(visible, dtype=torch.int32))
    kept[0, 2], kept[3, 1] = 10, -1
    d = {k: torch.from_numpy(v.copy()).cuda() for k, v in dst.items()}
    qsa.qsa_evict_compact(dims, 6, kept, torch.full((4,), 6, dtype=torch.int32, device="cuda"), qsa.QsaHistory.of(**s),
                          qsa.QsaHistory.of(**d), ws)
    assert qsa.qsa_check_errors(ws)[1] == qsa.QSA_DEVERR_ROW_RANGE
    for b, i in ((0, 2), (3, 1)):
        t0 = int(dst["key_offset"][b]) + 4 * i
        assert (d["idx_keys"][t0:t0 + 4] == 0).all() and (d["slot_map"][t0:t0 + 4] == -1).all()
        assert int(d["block_map"][int(dst["block_offset"][b]) + i]) == -1
        assert (d["pooled"][int(dst["pool_offset"][b]) + i] == 0).all()
        assert float(d["weights"][int(dst["weight_offset"][b]) + i]) == 0
        assert torch.equal(d["idx_keys"][t0 + 4:t0 + 8], s["idx_keys"][int(src["key_offset"][b]) + 4 * (i + 1):][:4])


# ---- together --------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("incremental", [False, True])
def test_decode_observe_evict_decode(fmt, incremental):
    """A bounded history as a program keeps it: groups pooled and coded, decode steps
    over the coded cache that accumulate what they attend to, an eviction, and
    decode steps over the moved history -- whose ID rows, outputs and weights are
    those of the plain forms over the kept groups."""
    torch = need_gpu()
    import oracle
    from top_group_sparse_gb300 import qsa
    from top_group_sparse_gb300 import workloads as wl
    visible, budget, keep, sink, recent = [2053, 9001, 7, 4002], 64, 300, 2, 8
    w = wl.make_workload("bounded", visible, idx_heads=8, idx_dim=64, q_heads=16, kv_heads=2, head_dim=128, seed=31,
                         slots="permutation", budget=budget)
    db = qsa.DeviceBatch(w)
    B = w.batch
    G = w.visible // 4
    h = ch.History(visible, q_heads=16, kv_heads=2, head_dim=128, fmt=fmt, seed=32)
    h.k, h.v, h.q = w.k_cache[w.slot_map], w.v_cache[w.slot_map], w.q   # the workload's rows in logical order
    h.weights0[:] = 0
    codes = torch.zeros(h.num_blocks, 2, 8 * 128, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(h.num_blocks, 2, 2, device="cuda")
    bm, bo = torch.from_numpy(h.block_map).cuda(), torch.from_numpy(h.group_offset).cuda()
    weights, wo = torch.from_numpy(h.weights0).cuda(), torch.from_numpy(h.weight_offset).cuda()
    cache = qsa.QsaCodedCache.of(codes, scales, bm, bo, fmt)
    ws = torch.zeros(qsa.qsa_coded_workspace_size(db.dims, False, True), dtype=torch.uint8, device="cuda")
    qsa.qsa_code_groups(db.dims, db.inputs, cache, torch.zeros(B, dtype=torch.int32, device="cuda"),
                        torch.from_numpy(G.astype(np.int32)).cuda(), int(G.max()), ws)
    pooled = po = None
    db.make_pooled_cache()
    db.pool_all()
    if incremental:
        pooled, po = db.pooled, db.pool_offset
    qsa.qsa_decode_coded(db.dims, db.inputs, cache, db.ids, db.n_ids, db.out, ws, pooled=pooled, pool_offset=po,
                         weights=weights, weight_offset=wo)
    assert qsa.qsa_check_errors(ws)[1] == 0
    ref = oracle.decode(w)
    rows = [ref["ids"][b, :ref["n_ids"][b]] for b in range(B)]
    for b in range(B):
        assert int(db.n_ids[b]) == len(rows[b]) and np.array_equal(db.ids[b, :len(rows[b])].cpu().numpy(), rows[b])
    want, share, tol, rel = ch.attention(h, rows)
    assert (np.abs(db.out.cpu().numpy() - want).max(axis=(1, 2)) <= tol).all()
    aw, at = ch.add_weights(h, share, rel)
    assert (np.abs(weights.cpu().numpy() - aw) <= at).all()

    # the eviction goes by the accumulated weights as they are
    kept = torch.full((B, keep), -1, dtype=torch.int32, device="cuda")
    n_kept = torch.zeros(B, dtype=torch.int32, device="cuda")
    qsa.qsa_evict_select(db.dims, db.visible, weights, wo, keep, sink, recent, kept, n_kept, ws)
    ks = ch.evict(visible, weights.cpu().numpy(), h.weight_offset, keep, sink, recent)
    after = [4 * len(k) + t % 4 for k, t in zip(ks, visible)]
    tok = np.concatenate([[0], np.cumsum(after)])[:-1]
    grp = np.concatenate([[0], np.cumsum([len(k) for k in ks])])[:-1]
    wgt = np.concatenate([[0], np.cumsum([-(-t // 4) for t in after])])[:-1]
    dev = {n: torch.from_numpy(a.astype(np.int64)).cuda() for n, a in (("tok", tok), ("grp", grp), ("wgt", wgt))}
    new = dict(idx_keys=torch.zeros(sum(after), 64, device="cuda"), key_offset=dev["tok"],
               pooled=torch.zeros(sum(map(len, ks)), 64, device="cuda"), pool_offset=dev["grp"],
               slot_map=torch.zeros(sum(after), dtype=torch.int32, device="cuda"), slot_offset=dev["tok"],
               block_map=torch.zeros(sum(map(len, ks)), dtype=torch.int32, device="cuda"), block_offset=dev["grp"],
               weights=torch.zeros(sum(-(-t // 4) for t in after), device="cuda"), weight_offset=dev["wgt"],
               visible=torch.zeros(B, dtype=torch.int32, device="cuda"))
    old = dict(idx_keys=db.idx_keys, key_offset=db.key_offset, pooled=db.pooled, pool_offset=db.pool_offset,
               slot_map=db.slot_map, slot_offset=db.slot_offset, block_map=bm, block_offset=bo, weights=weights,
               weight_offset=wo, visible=db.visible)
    qsa.qsa_evict_compact(db.dims, keep, kept, n_kept, qsa.QsaHistory.of(**old), qsa.QsaHistory.of(**new), ws)
    assert qsa.qsa_check_errors(ws)[1] == 0
    assert new["visible"].tolist() == after

    # a decode over the moved history: what the oracle says of a history of the kept tokens alone
    import dataclasses
    toks = [np.concatenate([(4 * k[:, None] + np.arange(4)).ravel(), np.arange(4 * (t // 4), t)]).astype(np.int64)
            for k, t in zip(ks, visible)]
    where = np.concatenate([w.key_offset[b] + toks[b] for b in range(B)])
    w2 = dataclasses.replace(w, idx_keys=w.idx_keys[where], slot_map=w.slot_map[where], key_offset=tok.astype(np.int64),
                             slot_offset=tok.astype(np.int64), visible=np.array(after, np.int32), max_visible=max(after))
    assert np.array_equal(new["idx_keys"].cpu().numpy(), w2.idx_keys) and np.array_equal(new["slot_map"].cpu().numpy(), w2.slot_map)
    inp = qsa.QsaInputs(q_idx=db.q_idx.data_ptr(), idx_keys=new["idx_keys"].data_ptr(), key_offset=dev["tok"].data_ptr(),
                        visible=new["visible"].data_ptr(), q=db.q.data_ptr(), k_cache=db.k_cache.data_ptr(),
                        v_cache=db.v_cache.data_ptr(), num_slots=w.num_slots, slot_map=new["slot_map"].data_ptr(),
                        slot_offset=dev["tok"].data_ptr())
    cache2 = qsa.QsaCodedCache.of(codes, scales, new["block_map"], dev["grp"], fmt)
    before = new["weights"].clone()
    qsa.qsa_decode_coded(db.dims, inp, cache2, db.ids, db.n_ids, db.out, ws, pooled=new["pooled"] if incremental else None,
                         pool_offset=dev["grp"] if incremental else None, weights=new["weights"], weight_offset=dev["wgt"])
    assert qsa.qsa_check_errors(ws)[1] == 0
    ref = oracle.decode(w2)
    K, V = h.coded()
    pick = np.concatenate([h.group_offset[b] + ks[b] for b in range(B)])
    h2 = ch.History(after, q_heads=16, kv_heads=2, head_dim=128, fmt=fmt, seed=33)
    h2.k, h2.v, h2.q = h.k[where], h.v[where], w.q
    rows = [ref["ids"][b, :ref["n_ids"][b]] for b in range(B)]
    for b in range(B):
        assert int(db.n_ids[b]) == len(rows[b]) and np.array_equal(db.ids[b, :len(rows[b])].cpu().numpy(), rows[b])
    want, share, tol, rel = ch.attention(h2, rows, coded=(K[pick], V[pick]))
    assert (np.abs(db.out.cpu().numpy() - want).max(axis=(1, 2)) <= tol).all()
    h2.weights0 = before.cpu().numpy()
    aw, at = ch.add_weights(h2, share, rel)
    assert (np.abs(new["weights"].cpu().numpy() - aw) <= at).all()


def test_the_whole_path_into_pinned_host_memory():
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    from top_group_sparse_gb300 import workloads as wl
    w = wl.make_workload("pinned", [9001, 0, 300, 2], idx_heads=4, idx_dim=32, q_heads=8, kv_heads=2, head_dim=64, seed=41,
                         slots="paged16", budget=40)
    db = qsa.DeviceBatch(w)
    G = (w.visible // 4).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(G)])[:-1].astype(np.int64)
    codes = torch.zeros(int(G.sum()), 2, 512, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(int(G.sum()), 2, 2, device="cuda")
    bm, bo = torch.arange(int(G.sum()), dtype=torch.int32, device="cuda"), torch.from_numpy(off).cuda()
    cache = qsa.QsaCodedCache.of(codes, scales, bm, bo, ch.INT8)
    qsa.qsa_code_groups(db.dims, db.inputs, cache, torch.zeros(4, dtype=torch.int32, device="cuda"), torch.from_numpy(G).cuda(),
                        int(G.max()), db.ws)
    qsa.qsa_decode_coded(db.dims, db.inputs, cache, db.ids, db.n_ids, db.out, db.ws)
    _, h_out = db.step_host_buffers()
    h_out.fill_(0xff)
    hi, hn, ho = db.host_outputs(h_out)
    qsa.qsa_decode_coded(db.dims, db.inputs, cache, hi, hn, ho, db.ws)
    torch.cuda.synchronize()
    assert db.check_errors()[1] == 0
    assert torch.equal(hn, db.n_ids.cpu()) and torch.equal(ho, db.out.cpu())
    for b in range(4):
        n = int(hn[b])
        assert torch.equal(hi[b, :n], db.ids[b, :n].cpu()) and (hi[b, n:] == -1).all()
    # the same rows and counts as the whole path over the f32 cache
    ids, n_ids = db.ids.clone(), db.n_ids.clone()
    db.decode()
    assert torch.equal(n_ids, db.n_ids) and torch.equal(ids, db.ids)
