"""Where the numbers of the coded cache are hardest to keep, against the plain forms
in 64 bits (tests/cache_helpers.py): scores that leave binary32."""
import numpy as np
import pytest

import cache_helpers as ch
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

HEADS = [(3, 3, 64), (8, 1, 64), (16, 2, 128), (12, 1, 128), (16, 1, 64)]


def _attend(h, rows, weights=False):
    """Output, accumulators and error word of one call over h's coded rows."""
    from top_group_sparse_gb300 import qsa
    t = ch.device(h, whole=rows is None, weights=weights)
    ch.fill_cache(h, t)
    ids, n_ids = (None, None) if rows is None else ch.rows_to_device(rows, 512)
    qsa.qsa_attend_coded(t["dims"], t["inputs"], t["cache"], ids, n_ids, t["out"], t["ws"],
                         weights=t["weights"] if weights else None,
                         weight_offset=t["weight_offset"] if weights else None)
    flags = qsa.qsa_check_errors(t["ws"])[1]
    return t["out"].cpu().numpy().astype(np.float64), t["weights"].cpu().numpy().astype(np.float64), flags


def _set_cache(h):
    h.k_cache[h.slot_map], h.v_cache[h.slot_map] = h.k, h.v


# ---- scores of -inf ----------------------------------------------------------------

@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("q_heads,kv,d", HEADS)
def test_scores_of_minus_infinity_get_no_weight(q_heads, kv, d, fmt, whole, shared):
    """q = 1e20 and K = -1: scores near -1e21, all equal, beside groups of K = -1e20 whose
    scores pass binary32's range -- each warp's first 16 tokens, some in the middle, and
    whole rows.  Those get exactly nothing; the others share the weight evenly, so that
    scores, however rounded, leave no error (30 * 2^-22: the weights' two parts and the
    sums, as in cache_helpers.attention).  A row without any other score gives zeros."""
    need_gpu()
    visible = [1028, 1024, 64, 16] if shared else [1028, 600, 64, 67, 3]
    h = ch.History(visible, q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=1, shared=shared)
    h.q[:] = 1e20
    h.k[:] = -1
    for t in [0] if shared else h.token_offset[:4]:
        h.k[t:t + 64] = -1e20
    for t in h.token_offset[:2]:
        h.k[t + 4 * 70:t + 4 * 74] = -1e20
    _set_cache(h)
    rows = None if whole else ch.some_rows(h, 512, 2)
    all_rows = rows or [np.arange(t) for t in visible]
    K, V = h.coded()
    share, want = [], np.zeros((h.B, q_heads, d))
    for b, row in enumerate(all_rows):
        w = np.zeros(-(-visible[b] // 4))
        p = (h.k[h.token_offset[b] + row, 0, 0] == -1).astype(np.float64)
        if p.any():
            p /= p.sum()
            np.add.at(w, row // 4, q_heads * p)
            n = len(row) // 4 * 4
            for hd in range(q_heads):
                v = np.concatenate([V[h.group_offset[b] + row[:n:4] // 4, hd // (q_heads // kv)].reshape(-1, d),
                                    h.v[h.token_offset[b] + row[n:], hd // (q_heads // kv)]])
                want[b, hd] = p @ v
        share.append(w)
    out, got, flags = _attend(h, rows, weights=True)
    assert flags == 0
    assert np.isfinite(out).all() and np.isfinite(got).all()
    assert np.abs(out - want).max() <= 30 * 2.0 ** -22 * np.abs(h.v).max()
    assert (out[2] == 0).all()
    w, wt = ch.add_weights(h, share, [30 * 2.0 ** -22] * h.B)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()
    untouched = w == h.weights0
    assert untouched.any() and (got[untouched] == h.weights0[untouched]).all()
