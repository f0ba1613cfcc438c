"""Histories that go on after an eviction: tokens appended behind the moved groups,
with accumulators in memory that was used before."""
import numpy as np
import pytest

import cache_helpers as ch
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
def test_accumulators_of_groups_that_start_after_a_move(fmt):
    """Moved into regions full of old numbers, then seven tokens appended one by one, each
    attended to with weights.  The caller sets a group's entry to 0 when its first token
    comes (behind a move without a raw tail that is entry n_kept); an incomplete group's
    goes on from what was moved with it.  What is behind the history stays as it was."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    visible, keep, steps, dirty = [40, 43, 64, 17, 24], 5, 7, 1e6
    B, room = len(visible), 4 * keep + 12
    # the history after the move, at its full room: the rows live in its caches
    h = ch.History([room] * B, q_heads=8, kv_heads=2, head_dim=64, fmt=fmt, seed=1)
    t = ch.device(h, whole=True, weights=True)
    r = np.random.RandomState(2)
    tok = np.concatenate([[0], np.cumsum(visible)]).astype(np.int64)
    grp = np.concatenate([[0], np.cumsum([v // 4 for v in visible])]).astype(np.int64)
    wgt = np.concatenate([[0], np.cumsum([-(-v // 4) for v in visible])]).astype(np.int64)
    w0 = r.rand(int(wgt[-1])).astype(np.float32)
    kept = ch.evict(visible, w0, wgt, keep, 1, 1)
    slots, blocks = np.zeros(int(tok[-1]), np.int32), np.zeros(int(grp[-1]), np.int32)
    acc, tol = np.full(h.n_weights, dirty), np.zeros(h.n_weights)
    now = np.array([4 * len(k) + v % 4 for k, v in zip(kept, visible)], np.int32)
    for b, v in enumerate(visible):
        n, to = len(kept[b]), h.token_offset[b]
        rows = np.concatenate([(4 * kept[b][:, None] + np.arange(4)).ravel(), np.arange(v // 4 * 4, v)]).astype(np.int64)
        slots[tok[b] + rows] = h.slot_map[to:to + len(rows)]
        blocks[grp[b] + kept[b]] = h.block_map[h.group_offset[b]:h.group_offset[b] + n]
        moved = np.concatenate([kept[b], [v // 4]]) if v % 4 else kept[b]
        acc[h.weight_offset[b]:h.weight_offset[b] + len(moved)] = w0[wgt[b] + moved]

    def put(a, dtype=None):
        return torch.from_numpy(np.ascontiguousarray(a if dtype is None else a.astype(dtype))).cuda()

    src = dict(slot_map=put(slots), slot_offset=put(tok[:-1]), block_map=put(blocks), block_offset=put(grp[:-1]),
               weights=put(w0), weight_offset=put(wgt[:-1]), visible=put(np.array(visible, np.int32)))
    dst = dict(slot_map=torch.full_like(t["slot_map"], -7), slot_offset=t["token_offset"],
               block_map=torch.full_like(t["block_map"], -7), block_offset=t["group_offset"],
               weights=torch.full((h.n_weights,), dirty, device="cuda"), weight_offset=t["weight_offset"],
               visible=torch.full((B,), -7, dtype=torch.int32, device="cuda"))
    kt = np.full((B, keep), -1, np.int32)
    for b, k in enumerate(kept):
        kt[b, :len(k)] = k
    dims = qsa.make_dims(B, 8, 64, 8, 2, 64, max_visible=max(visible), scale=h.scale)
    qsa.qsa_evict_compact(dims, keep, put(kt), put(np.array([len(k) for k in kept], np.int32)), qsa.QsaHistory.of(**src),
                          qsa.QsaHistory.of(**dst), t["ws"])
    assert dst["visible"].tolist() == now.tolist()
    assert np.array_equal(dst["weights"].cpu().numpy(), acc.astype(np.float32))

    inp = qsa.QsaInputs(visible=dst["visible"].data_ptr(), q=t["q"].data_ptr(), k_cache=t["k_cache"].data_ptr(),
                        v_cache=t["v_cache"].data_ptr(), num_slots=h.num_slots, slot_map=dst["slot_map"].data_ptr(),
                        slot_offset=t["token_offset"].data_ptr())
    cache = qsa.QsaCodedCache.of(t["codes"], t["scales"], dst["block_map"], t["group_offset"], fmt)
    qsa.qsa_code_groups(t["dims"], inp, cache, put(0 * now), put(now // 4), keep, t["ws"])
    for _ in range(steps):
        for b in range(B):
            T, to, wo = int(now[b]), int(h.token_offset[b]), int(h.weight_offset[b])
            if T % 4 == 0:
                dst["weights"][wo + T // 4] = 0
                acc[wo + T // 4] = 0
            dst["slot_map"][to + T] = int(h.slot_map[to + T])
            if T % 4 == 3:
                at = int(h.group_offset[b]) + T // 4
                dst["block_map"][at] = int(h.block_map[at])
        now += 1
        dst["visible"].copy_(put(now))
        done = now % 4 == 0
        qsa.qsa_code_groups(t["dims"], inp, cache, put(np.where(done, now // 4 - 1, 0), np.int32),
                            put(np.where(done, now // 4, 0), np.int32), 1, t["ws"])
        qsa.qsa_attend_coded(t["dims"], inp, cache, None, None, t["out"], t["ws"], weights=dst["weights"],
                             weight_offset=t["weight_offset"])
        assert qsa.qsa_check_errors(t["ws"])[1] == 0
        h.visible = now
        h.weights0 = acc
        ref, share, out_tol, rel = ch.attention(h)
        assert (np.abs(t["out"].cpu().numpy() - ref).max(axis=(1, 2)) <= out_tol).all()
        acc, wt = ch.add_weights(h, share, rel)
        tol += wt
    got = dst["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - acc) <= tol).all(), np.abs(got - acc).max()
    for b in range(B):
        lo, hi = int(h.weight_offset[b]), int(h.weight_offset[b]) + room // 4
        n = -(-int(now[b]) // 4)
        assert (got[lo:lo + n] < 8 * (steps + 1)).all() and (got[lo + n:hi] == dirty).all()
