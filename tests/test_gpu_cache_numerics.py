"""Where the numbers of the coded cache are hardest to keep, against the plain forms
in 64 bits (tests/cache_helpers.py): scores that leave binary32 or come near, values of
neighbouring groups whose sizes differ, zeros with a sign, long shared sums."""
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


# ---- values of neighbouring groups that differ in size -----------------------------------

def _bound(h, b, hd, row, K, V, same_scores=False):
    """(output of head hd over a row of whole groups, its tolerance per dim) in 64 bits.

    A weight p * sV enters as two 16-bit floats under a power of two that brings the
    largest of its head's in the step (four consecutive groups of the row) to 2^12 or
    more: it keeps 22 bits, or 2^-25 of that scale, i.e. 2^-37 of the largest.  All other
    errors are relative to the sum of |p v| in the dim itself: 2^-22 * (14 S + 30) as
    derived in cache_helpers.attention, without S where the scores' errors cancel."""
    kv = hd // (h.q_heads // h.kv_heads)
    g = h.group_offset[b] + row[::4] // 4
    k, v = K[g, kv].reshape(-1, h.d), V[g, kv].reshape(-1, h.d)
    q = h.q[b, hd].astype(np.float64)
    x = (k @ q) * h.scale
    S = 0.0 if same_scores else float((np.abs(k) @ np.abs(q)).max()) * h.scale
    p = np.exp(x - x.max())
    p /= p.sum()
    sv = ch.encode(h.v[h.token_offset[b] + 4 * (row[::4] // 4)[:, None] + np.arange(4)][:, :, kv], h.fmt)[1].astype(np.float64)
    w = p * np.repeat(sv, 4)
    pad = -len(w) % 16
    step = np.concatenate([w, np.zeros(pad)]).reshape(-1, 16).max(axis=1)
    codes = np.abs(v) / np.repeat(np.where(sv > 0, sv, 1), 4)[:, None]
    tol = 2.0 ** -22 * (14 * S + 30) * (p @ np.abs(v)) + 2.0 ** -37 * (np.repeat(step, 16)[:len(w)] @ codes)
    return p @ v, tol


def _check_per_dim(h, rows, whole, same_scores):
    K, V = h.coded()
    out, _, flags = _attend(h, None if whole else rows)
    assert flags == 0 and np.isfinite(out).all()
    for b in range(h.B):
        for hd in range(h.q_heads):
            want, tol = _bound(h, b, hd, rows[b], K, V, same_scores)
            err = np.abs(out[b, hd] - want)
            assert (err <= tol).all(), (b, hd, (err / tol).max(), (err / np.abs(want).max()).max())


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("q_heads,kv,d", HEADS)
@pytest.mark.parametrize("exponent", [0, 80, -80])
def test_a_small_group_that_takes_the_weight_beside_large_ones(exponent, q_heads, kv, d, fmt, whole):
    """One group takes the weight, its values 2^-4 .. 2^-32 of its step neighbours', whose
    weights are below 2^-60 of its own.  Its four tokens have one value, so the output is
    that value whatever the scores' errors do to their weights."""
    need_gpu()
    r = np.random.RandomState(3)
    ratios = [4, 12, 16, 20, 24, 32]
    groups = [40, 77, 100, 64, 300, 13]
    h = ch.History([4 * g for g in groups], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=4)
    u = r.choice([-1.0, 1.0], (kv, d)).astype(np.float32)
    h.q[:] = np.repeat(u, q_heads // kv, axis=0)[None]
    h.k[:] = -3 * u
    for b, (n, ratio) in enumerate(zip(groups, ratios)):
        t = h.token_offset[b] + 4 * r.randint(n)
        h.k[t:t + 4] = 3 * u
        h.v[t:t + 4] = h.v[t] * np.float32(2.0 ** -ratio)
    h.v *= np.float32(2.0 ** exponent)
    _set_cache(h)
    _check_per_dim(h, [np.arange(4 * g) for g in groups], whole, True)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("q_heads,kv,d", HEADS)
def test_groups_that_weigh_the_more_the_smaller_they_are(q_heads, kv, d, fmt, whole):
    """Values of 2^-r and weights near 2^r, r from 0 to 24 from group to group (and some
    groups of zeros): all contribute alike."""
    need_gpu()
    r = np.random.RandomState(5)
    groups = [130, 512, 7, 64]
    h = ch.History([4 * g for g in groups], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=6)
    u = r.choice([-1.0, 1.0], (kv, d)).astype(np.float32)
    h.q[:] = np.repeat(u, q_heads // kv, axis=0)[None] * (0.75 + 0.5 * r.rand(1, q_heads, 1)).astype(np.float32)
    e = np.repeat(r.randint(0, 25, sum(groups)), 4)
    h.k[:] = u * (e * np.log(2) / (h.scale * d))[:, None, None].astype(np.float32)
    h.v *= (2.0 ** -e)[:, None, None].astype(np.float32)
    h.v[np.repeat(r.rand(sum(groups)) < 0.1, 4)] = 0
    _set_cache(h)
    _check_per_dim(h, [np.arange(4 * g) for g in groups], whole, False)


# ---- scores whose neighbours are 16 apart -------------------------------------------------

@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("q_heads,kv,d", [(8, 1, 64), (16, 1, 64), (16, 2, 128), (16, 1, 128)])
def test_scores_near_two_to_the_27(q_heads, kv, d, fmt, whole):
    """Scores (base 2) between 2^27 and 2^28, where binary32's numbers are 16 apart and a
    running maximum plus 8 may round to the next of them, so that a weight of 2^16
    follows without a new maximum.  K scales that differ in the last bit give scores one
    number apart.  What such scores' weights are is up to their rounding; the outputs
    are averages of values all the same: each lies between the least and the largest of
    its dim (30 * 2^-22: the sums' own rounding)."""
    need_gpu()
    r = np.random.RandomState(9)
    G = 300
    h = ch.History([4 * G], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=10)
    amp = 2.0 ** 27.3 / (d * h.scale * 1.4427) * (1 + np.arange(q_heads) / 32)
    h.q[:] = amp[None, :, None].astype(np.float32)
    up = np.where(np.arange(G) < 16, 0, r.randint(0, 2, G)).astype(np.uint32)
    h.k[:] = np.repeat((np.float32(1).view(np.uint32) + up).view(np.float32), 4)[:, None, None]
    _set_cache(h)
    rows = None if whole else [np.arange(4 * G)]
    out, _, flags = _attend(h, rows)
    assert flags == 0 and np.isfinite(out).all()
    V = h.coded()[1]
    for hd in range(q_heads):
        v = V[:, hd // (q_heads // kv)].reshape(-1, d)
        slack = 30 * 2.0 ** -22 * np.abs(v).max()
        assert (out[0, hd] <= v.max(axis=0) + slack).all() and (out[0, hd] >= v.min(axis=0) - slack).all()


# ---- zeros with a sign --------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_code_bytes_equal_the_definition_with_signed_zeros(fmt, d):
    """The bytes, not the numbers they stand for: an e4m3 code has the sign of its value,
    -0 and what rounds to it included, whatever the group's scale (scales on both sides
    of 2^-90, below which the quotient is computed in another way)."""
    need_gpu()
    r = np.random.RandomState(7)
    exponents = [-140, -126, -100, -92, -91, -90, -89, -88, -60, -1, 0, 1, 60, 120]
    h = ch.History([4 * len(exponents)], q_heads=2, kv_heads=2, head_dim=d, fmt=fmt, seed=8)
    for x in (h.k, h.v):
        small = r.rand(*x.shape)
        x[small < 0.3] = 0.0
        x[small < 0.2] *= np.float32(1e-30)
        x[(small > 0.3) & (small < 0.4)] *= np.float32(1e-4)
        x[(small > 0.4) & (small < 0.5)] *= np.float32(1e-36)
        x *= np.repeat(2.0 ** np.array(exponents) * ch.QMAX[fmt], 4)[:, None, None].astype(np.float64) / 8
        x[r.rand(*x.shape) < 0.5] *= -1
    assert np.signbit(h.k[h.k == 0]).any() and not np.signbit(h.k[h.k == 0]).all()
    _set_cache(h)
    t = ch.device(h)
    t["codes"].fill_(0x5a)
    ch.fill_cache(h, t)
    raw = t["codes"].cpu().numpy()[h.block_map]
    n = len(exponents)
    k = raw[:, :, :4 * d].reshape(n, 2, d // 64, 4, 64).transpose(0, 1, 3, 2, 4).reshape(n, 2, 4, d)
    v = raw[:, :, 4 * d:].reshape(n, 2, d, 4).transpose(0, 1, 3, 2)
    table = ch.e4m3_table()[:0x7f]
    for src, got in ((h.k, k), (h.v, v)):
        x = src.reshape(n, 4, 2, d).transpose(0, 2, 1, 3)
        c, s = ch.encode(x, fmt)
        if fmt == ch.INT8:
            want = c.astype(np.int8).view(np.uint8)
        else:
            want = np.searchsorted(table, np.abs(c)).astype(np.uint8)
            assert np.array_equal(table[want], np.abs(c))
            want = np.where(np.signbit(x) & (s > 0)[..., None, None], want | 0x80, want)
        assert np.array_equal(got, want)


# ---- several queries of one long history ----------------------------------------------------

@pytest.mark.parametrize("fmt,q_heads,kv,d", [(ch.E4M3, 8, 2, 64), (ch.INT8, 16, 1, 128)])
def test_queries_of_one_long_history_over_all_of_it(fmt, q_heads, kv, d):
    """Five queries of one history on both sides of the changes of the run length, with
    the weights they add to its accumulators."""
    need_gpu()
    visible = [4 * 1024 + 3, 4 * 1025, 4 * 4096 + 1, 4 * 4097 + 2, 4 * 4400 + 3]
    h = ch.History(visible, q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=11, shared=True)
    out, got, flags = _attend(h, None, weights=True)
    assert flags == 0
    ref, share, tol, rel = ch.attention(h)
    assert (np.abs(out - ref).max(axis=(1, 2)) <= tol).all()
    w, wt = ch.add_weights(h, share, rel)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()
