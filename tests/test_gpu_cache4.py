"""The K/V cache in 4 bits on the GPU: coding, reading back and the attention over
it, against the plain forms in 64 bits (tests/cache4_helpers.py, cache_helpers.py).

The tolerance of cache_helpers.attention counts what the 8-bit kernel rounds; this
one rounds the same at the same places: a code times its tile scale is exact (so
are int4's eighths), a chain of the first product covers d dims in at most eight
accumulations, and one of the second 32 tokens in two instead of 16 in one, 2 * 2^-23
of the sum more, which the 30 * 2^-22 of that derivation covers."""
import numpy as np
import pytest

import cache4_helpers as c4
import cache_helpers as ch
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

FORMATS = [c4.E2M1, c4.INT4]
LENGTHS = [0, 1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 35, 63, 65, 127, 131, 259, 509, 1027, 2051, 4096, 4099, 9001]
HEADS = [(1, 1, 64), (2, 2, 64), (8, 2, 64), (16, 2, 128), (16, 1, 128), (10, 2, 128), (12, 1, 64), (9, 1, 128), (24, 8, 128)]


def _flags(t):
    from top_group_sparse_gb300 import qsa
    return qsa.qsa_check_errors(t["ws"])[1]


def _attend(t, ids=None, n_ids=None, weights=False, stream=None):
    from top_group_sparse_gb300 import qsa
    qsa.qsa_attend_coded(t["dims"], t["inputs"], t["cache"], ids, n_ids, t["out"], t["ws"],
                         weights=t["weights"] if weights else None,
                         weight_offset=t["weight_offset"] if weights else None, stream=stream)
    return t["out"]


def _close(h, got, ref, tol):
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    for b in range(h.B):
        err = np.abs(got[b] - ref[b]).max(initial=0.0)
        assert err <= tol[b], f"query {b} (T {h.visible[b]}): {err:.3e} > {tol[b]:.3e}"


def _equals_the_coding(h, t):
    """Every group of every history is coded as the definition says; returns which blocks were written."""
    raw, s = t["codes"].cpu().numpy(), t["scales"].cpu().numpy()
    got = c4.unpack(raw, h.d, h.fmt)
    done = np.zeros(h.num_blocks, bool)
    for b, T in enumerate(h.visible):
        n = int(T) // 4
        blk = h.block_map[h.group_offset[b]:h.group_offset[b] + n]
        done[blk] = True
        for i, src in enumerate((h.k, h.v)):
            x = src[h.token_offset[b]:h.token_offset[b] + 4 * n].reshape(n, 4, h.kv_heads, h.d).transpose(0, 2, 1, 3)
            code, tile, scale = c4.encode(x, h.fmt)
            assert np.array_equal(s[blk, :, i], scale, equal_nan=True)
            assert np.array_equal(got[2 + i][blk], tile)
            assert np.array_equal(got[i][blk], code)
    return done


# ---- coding and reading back -----------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kv,d", [(1, 64), (3, 64), (2, 128), (5, 128)])
def test_codes_and_scales_equal_the_definition(fmt, kv, d):
    need_gpu()
    h = c4.History([0, 3, 4, 7, 64, 1029, 517], q_heads=kv, kv_heads=kv, head_dim=d, fmt=fmt, seed=3)
    r = np.random.RandomState(1)
    h.k *= np.exp(3 * r.randn(len(h.k), 1, 1)).astype(np.float32)
    h.k *= np.where(r.rand(kv, d) > 0.9, 30, 1).astype(np.float32)     # wide channels
    h.v[::5, :, ::3] = 0
    h.v[1::5, :, ::7] *= -1e-6                                         # tiles far below their group
    h.set_cache()
    t = c4.device(h)
    t["codes"].fill_(0x5a)
    t["scales"].fill_(-3.0)
    ch.fill_cache(h, t)
    assert _flags(t) == 0
    done = _equals_the_coding(h, t)
    assert (t["codes"].cpu().numpy()[~done] == 0x5a).all() and (t["scales"].cpu().numpy()[~done] == -3.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_coding_of_extreme_groups(fmt, d):
    """Zero, tiny, subnormal, huge, infinite and NaN groups, each beside an ordinary one; tiles whose
    scales are subnormal e4m3 numbers or none."""
    need_gpu()
    vals = [0.0, 1e-45, 1e-38, 3e-35, 4e-35, 1e-30, 1e-22, 3e-21, 3.3e38, np.inf, -np.inf, np.nan, 1.0, -2.0 ** 14, 2.0 ** 19, 2.0 ** 20]
    h = c4.History([4 * len(vals)], q_heads=2, kv_heads=2, head_dim=d, fmt=fmt, seed=5)
    for i, v in enumerate(vals):
        if v == 0 or abs(v) < 1e-20:
            h.k[4 * i:4 * i + 4] = (np.random.RandomState(i).rand(4, 2, d) * v).astype(np.float32)
        h.k[4 * i + i % 4, 0, (7 * i) % d] = v     # head 0 only
        h.v[4 * i + 3, 1, (5 * i) % d] = v
    h.set_cache()
    t = c4.device(h)
    ch.fill_cache(h, t)
    assert _flags(t) == 0
    _equals_the_coding(h, t)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("log2_scale", [-117, -81, -79, -40, 0, 3, 100])
def test_codes_next_to_the_borders_between_codes(fmt, log2_scale):
    """Values at, and one or two units beside, the middle of two codes of their tile, and tiles
    at the middle of two tile scales: the rounded quotient decides."""
    need_gpu()
    r = np.random.RandomState(8)
    n, d = 300, 64
    h = c4.History([4 * n], q_heads=1, kv_heads=1, head_dim=d, fmt=fmt, seed=9)
    grid = c4.e2m1_table()[:8] if fmt == c4.E2M1 else np.arange(8.0)
    mid = (grid[1:] + grid[:-1]) / 2
    scales = np.unique(np.abs(ch.e4m3_table()[:0x7f]))
    for a in (h.k, h.v):
        amax = (2.0 ** log2_scale * (1 + r.rand(n))).astype(np.float32)
        s = (amax * np.float32(1.0 / (448 * c4.TOP[fmt]))).astype(np.float64)
        # the tile's scale is t (or between two), so its largest value is c * t * s
        at = r.randint(20, len(scales) - 1, (n, d // 4))
        t = np.where(r.rand(n, d // 4) < 0.5, scales[at], (scales[at] + scales[at + 1]) / 2)
        near = c4.nearest_e4m3(t)
        x = mid[r.randint(0, len(mid), (n, 4, d // 4, 4))] * (near * s[:, None])[:, None, :, None]
        x[np.arange(n)[:, None], r.randint(0, 4, (n, d // 4)), np.arange(d // 4), r.randint(0, 4, (n, d // 4))] = c4.TOP[fmt] * t * s[:, None]
        x = x.astype(np.float32).reshape(n, 4 * d)
        x = (x.view(np.int32) + r.randint(-2, 3, x.shape).astype(np.int32)).view(np.float32) * r.choice([-1, 1], x.shape).astype(np.float32)
        x = np.clip(x, -amax[:, None], amax[:, None])
        x[np.arange(n), r.randint(0, 4 * d, n)] = amax
        a[:] = x.reshape(4 * n, 1, d)
    h.set_cache()
    t = c4.device(h)
    ch.fill_cache(h, t)
    assert _flags(t) == 0
    _equals_the_coding(h, t)


@pytest.mark.parametrize("fmt", FORMATS)
def test_coding_flags_and_skips_what_is_out_of_range(fmt):
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = c4.History([64, 64, 64], q_heads=2, kv_heads=2, head_dim=64, fmt=fmt, seed=6)
    t = c4.device(h)
    for lo, hi, most in (([-1, 0, 0], [1, 0, 0], 1), ([0, 5, 0], [0, 4, 0], 1), ([0, 0, 16], [0, 0, 17], 1), ([0, 0, 0], [0, 2, 0], 1)):
        t["codes"].fill_(9)
        qsa.qsa_code_groups(t["dims"], t["inputs"], t["cache"], torch.tensor(lo, dtype=torch.int32, device="cuda"),
                            torch.tensor(hi, dtype=torch.int32, device="cuda"), most, t["ws"])
        assert _flags(t) == qsa.QSA_DEVERR_VISIBLE_RANGE
        assert (t["codes"] == 9).all()
    bm = t["block_map"].clone()
    t["block_map"][3] = h.num_blocks
    t["block_map"][4] = -1
    t["slot_map"][8] = h.num_slots
    t["slot_map"][9] = -7
    t["codes"].fill_(9)
    ch.fill_cache(h, t)
    assert _flags(t) == qsa.QSA_DEVERR_SLOT_RANGE
    raw = t["codes"].cpu().numpy()
    K = c4.unpack(raw, 64, fmt)[0]
    for g in range(48):
        if g in (3, 4):
            assert (raw[int(bm[g])] == 9).all()
            continue
        x = h.k[4 * g:4 * g + 4].copy()
        if g == 2:
            x[:2] = 0
        assert np.array_equal(K[int(bm[g])], c4.encode(x.transpose(1, 0, 2), fmt)[0]), g


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8] + FORMATS)
@pytest.mark.parametrize("kv,d", [(1, 64), (3, 64), (2, 128), (5, 128)])
def test_reading_back_gives_the_values_that_blocks_stand_for(fmt, kv, d):
    """Into rows of another cache and another slot map: what is read is the product, rounded once;
    what is not of the ranges stays."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    four = fmt in FORMATS
    h = (c4 if four else ch).History([0, 3, 4, 70, 517, 1031], q_heads=kv, kv_heads=kv, head_dim=d, fmt=fmt, seed=41)
    h.k[h.token_offset[3] + 5, 0, 1] = np.nan   # group 1 of query 3, head 0: a scale that is NaN
    h.k[h.token_offset[4]:h.token_offset[4] + 4] *= np.float32(2.0 ** 90)
    h.v[h.token_offset[4] + 4:h.token_offset[4] + 8] *= np.float32(2.0 ** -100)
    h.k_cache[h.slot_map], h.v_cache[h.slot_map] = h.k, h.v
    t = (c4 if four else ch).device(h)
    ch.fill_cache(h, t)
    r = np.random.RandomState(42)
    slots = r.permutation(h.num_slots + 9)[:len(h.slot_map)].astype(np.int32)
    kb, vb = (torch.full((h.num_slots + 9, kv, d), -5.0, device="cuda") for _ in range(2))
    lo = np.array([0, 0, 0, 0, 3, 100], np.int32)
    hi = np.array([0, 0, 1, 17, 129, 257], np.int32)
    sm = torch.from_numpy(slots).cuda()
    inp = qsa.QsaInputs(k_cache=kb.data_ptr(), v_cache=vb.data_ptr(), num_slots=h.num_slots + 9, slot_map=sm.data_ptr(),
                        slot_offset=t["token_offset"].data_ptr())
    ws = torch.zeros(qsa.QSA_ROWS_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    lo_t, hi_t = torch.from_numpy(lo).cuda(), torch.from_numpy(hi).cuda()
    qsa.qsa_read_groups(t["dims"], inp, t["cache"], lo_t, hi_t, int((hi - lo).max()), ws)
    assert qsa.qsa_check_errors(ws) == (0, 0)
    want = [np.full((h.num_slots + 9, kv, d), -5.0, np.float32) for _ in range(2)]
    for b in range(h.B):
        n = int(hi[b] - lo[b])
        at = int(h.token_offset[b]) + 4 * int(lo[b])
        for src, dst in ((h.k, want[0]), (h.v, want[1])):
            x = src[at:at + 4 * n].reshape(n, 4, kv, d).transpose(0, 2, 1, 3)
            if four:
                c, tile, s = c4.encode(x, fmt)
                c = c * np.repeat(tile, 4, axis=-1)[..., None, :]
            else:
                c, s = ch.encode(x, fmt)
            with np.errstate(invalid="ignore"):
                y = (c * s.astype(np.float64)[..., None, None]).astype(np.float32)
            dst[slots[at:at + 4 * n]] = y.transpose(0, 2, 1, 3).reshape(-1, kv, d)
    assert np.array_equal(kb.cpu().numpy(), want[0], equal_nan=True) and np.isnan(want[0]).sum() == 4 * d
    assert np.array_equal(vb.cpu().numpy(), want[1])


def test_reading_flags_and_skips_what_is_out_of_range():
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = c4.History([64, 64], q_heads=2, kv_heads=2, head_dim=64, fmt=c4.INT4, seed=43)
    t = c4.device(h)
    ch.fill_cache(h, t)
    kb, vb = (torch.full((h.num_slots, 2, 64), -5.0, device="cuda") for _ in range(2))
    inp = qsa.QsaInputs(k_cache=kb.data_ptr(), v_cache=vb.data_ptr(), num_slots=h.num_slots,
                        slot_map=t["slot_map"].data_ptr(), slot_offset=t["token_offset"].data_ptr())
    for lo, hi in (([-1, 0], [0, 0]), ([0, 3], [0, 2]), ([0, 16], [0, 17]), ([0, 0], [3, 0])):
        qsa.qsa_read_groups(t["dims"], inp, t["cache"], torch.tensor(lo, dtype=torch.int32, device="cuda"),
                            torch.tensor(hi, dtype=torch.int32, device="cuda"), 2, t["ws"])
        assert _flags(t) == qsa.QSA_DEVERR_VISIBLE_RANGE
        assert (kb == -5).all() and (vb == -5).all()
    sl = h.slot_map
    t["block_map"][1] = h.num_blocks        # zero rows
    t["block_map"][2] = -1
    t["slot_map"][12] = -1                  # skipped
    t["slot_map"][13] = h.num_slots
    qsa.qsa_read_groups(t["dims"], inp, t["cache"], t["lo"], t["hi"], 16, t["ws"])
    assert _flags(t) == qsa.QSA_DEVERR_SLOT_RANGE
    k = kb.cpu().numpy()
    assert (k[sl[4:12]] == 0).all() and (k[sl[12:14]] == -5).all()
    assert (np.abs(k[sl[14:]]).max(axis=(1, 2)) > 0.1).all() and (np.abs(k[sl[:4]]).max(axis=(1, 2)) > 0.1).all()
    assert (vb.cpu().numpy()[sl[4:12]] == 0).all()


# ---- attention ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_heads,kv,d", HEADS)
def test_attention_over_whole_histories(fmt, q_heads, kv, d):
    need_gpu()
    h = c4.History(LENGTHS, q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=11)
    t = c4.device(h, whole=True, weights=True)
    ch.fill_cache(h, t)
    ref, share, tol, rel = ch.attention(h)
    _close(h, _attend(t), ref, tol)
    assert _flags(t) == 0
    first = t["out"].clone()
    _attend(t, weights=True)
    assert _flags(t) == 0
    assert (t["out"] == first).all()
    w, wt = ch.add_weights(h, share, rel)
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()


@pytest.mark.parametrize("fmt,q_heads", [(c4.E2M1, 3), (c4.INT4, 12)])
def test_attention_over_long_histories(fmt, q_heads):
    """Rows on both sides of each change of the run length, whose runs take several segments."""
    need_gpu()
    h = c4.History([4 * 4097 + 1, 5, 4 * 4096, 4 * 65537 + 2, 4 * 131073 + 3], q_heads=q_heads, kv_heads=1, head_dim=64, fmt=fmt,
                   seed=27)
    t = c4.device(h, whole=True, weights=True)
    ch.fill_cache(h, t)
    ref, share, tol, rel = ch.attention(h)
    # (512/8 slices of runs and 64 steps a warp: more additions than the bound of shorter rows counts)
    vmax = max(float(np.abs(h.v).max()), 1.0) * 1.1
    _close(h, _attend(t, weights=True), ref, tol + vmax * 192 * 2.0 ** -24)
    assert _flags(t) == 0
    w, wt = ch.add_weights(h, share, [r + 192 * 2.0 ** -24 for r in rel])
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()


@pytest.mark.parametrize("budget", [512, 32, 5, 1])
@pytest.mark.parametrize("fmt,q_heads,kv,d", [(c4.E2M1, 16, 2, 128), (c4.INT4, 8, 2, 64), (c4.INT4, 16, 1, 128), (c4.E2M1, 3, 3, 64)])
def test_attention_over_selected_rows(budget, fmt, q_heads, kv, d):
    need_gpu()
    h = c4.History([0, 1, 3, 4, 6, 70, 128, 131, 2051, 9002, 4097], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=12)
    rows = ch.some_rows(h, budget, 13)
    t = c4.device(h, budget=budget, weights=True)
    ch.fill_cache(h, t)
    ids, n = ch.rows_to_device(rows, budget)
    ref, share, tol, rel = ch.attention(h, rows)
    _close(h, _attend(t, ids, n), ref, tol)
    first = t["out"].clone()
    _attend(t, ids, n, weights=True)
    assert _flags(t) == 0
    assert (t["out"] == first).all()
    w, wt = ch.add_weights(h, share, rel)
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_of_a_shared_history(whole, fmt):
    torch = need_gpu()
    vis = [989 + i for i in range(39)]
    h = c4.History(vis, q_heads=8, kv_heads=2, head_dim=64, fmt=fmt, seed=14, shared=True)
    t = c4.device(h, budget=64, whole=whole, weights=True)
    ch.fill_cache(h, t)
    rows = None if whole else ch.some_rows(h, 64, 15)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 64)
    ref, share, tol, rel = ch.attention(h, rows)
    _close(h, _attend(t, ids, n, weights=True), ref, tol)
    assert _flags(t) == 0
    w, wt = ch.add_weights(h, share, rel)
    assert (np.abs(t["weights"].cpu().numpy() - w) <= wt).all()
    again = t["weights"].clone()
    for _ in range(3):
        t["weights"].copy_(torch.from_numpy(h.weights0))
        _attend(t, ids, n, weights=True)
        assert torch.equal(t["weights"], again)


@pytest.mark.parametrize("fmt,q_heads,kv,d", [(c4.E2M1, 16, 2, 128), (c4.INT4, 12, 1, 64)])
def test_an_output_does_not_depend_on_the_batch_or_the_workspace(fmt, q_heads, kv, d):
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = c4.History([4101, 77, 9001, 0, 640, 35], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=16)
    t = c4.device(h, whole=True)
    ch.fill_cache(h, t)
    out = _attend(t).clone()
    assert torch.equal(_attend(t), out)
    for b in range(h.B):
        dims = qsa.make_dims(1, 8, 64, q_heads, kv, d, max_visible=int(h.visible[b]) + 1000 * b, scale=h.scale)
        ws = torch.full((qsa.qsa_coded_workspace_size(dims, True),), 0xa5, dtype=torch.uint8, device="cuda")
        ws[:qsa.QSA_ROWS_WORKSPACE_BYTES] = 0   # the error word alone has to start clean
        inp = qsa.QsaInputs(visible=t["visible"][b:].data_ptr(), q=t["q"][b:].data_ptr(), k_cache=t["k_cache"].data_ptr(),
                            v_cache=t["v_cache"].data_ptr(), num_slots=h.num_slots, slot_map=t["slot_map"].data_ptr(),
                            slot_offset=t["token_offset"][b:].data_ptr())
        cache = qsa.QsaCodedCache.of(t["codes"], t["scales"], t["block_map"], t["group_offset"][b:], h.fmt)
        one = torch.full((1, q_heads, d), float("nan"), device="cuda")
        qsa.qsa_attend_coded(dims, inp, cache, None, None, one, ws)
        assert torch.equal(one[0], out[b]), b


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_heads", [8, 16])
def test_wide_ranges_of_scales_and_scores(fmt, q_heads):
    """Scores spread over hundreds, queries and groups whose sizes differ by 2^40, zero queries."""
    need_gpu()
    h = c4.History([2000, 2000, 333, 1200], q_heads=q_heads, kv_heads=1, head_dim=128, fmt=fmt, seed=17)
    r = np.random.RandomState(18)
    h.q[0] *= 60
    h.q[2] = 0
    h.q[3] *= 2.0 ** -20
    for x in (h.k, h.v):
        x[h.token_offset[3]:] *= 2.0 ** 20
    h.v[:2000] *= np.repeat(2.0 ** r.randint(-20, 20, 500), 4)[:, None, None].astype(np.float32)
    h.set_cache()
    t = c4.device(h, whole=True)
    ch.fill_cache(h, t)
    ref, _, tol, _ = ch.attention(h)
    _close(h, _attend(t), ref, tol)
    assert _flags(t) == 0


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_heads,kv,d", [(3, 3, 64), (8, 1, 64), (16, 2, 128), (12, 1, 128), (16, 1, 64)])
def test_scores_of_minus_infinity_and_equal_huge_ones(q_heads, kv, d, fmt, whole):
    """q = 1e20 and K = -1: scores near -1e21, all equal, beside groups of K = -1e20 whose scores
    pass binary32's range.  Those get exactly nothing; the others share the weight evenly, so that
    scores, however rounded, leave no error (30 * 2^-22).  A row without any other score gives zeros."""
    need_gpu()
    visible = [1028, 600, 64, 67, 3]
    h = c4.History(visible, q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=1)
    h.q[:] = 1e20
    h.k[:] = -1
    for t0 in h.token_offset[:4]:
        h.k[t0:t0 + 64] = -1e20
    for t0 in h.token_offset[:2]:
        h.k[t0 + 4 * 70:t0 + 4 * 74] = -1e20
    h.set_cache()
    rows = None if whole else ch.some_rows(h, 512, 2)
    all_rows = rows or [np.arange(v) for v in visible]
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
    t = c4.device(h, whole=whole, weights=True)
    ch.fill_cache(h, t)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 512)
    out = _attend(t, ids, n, weights=True).cpu().numpy()
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert _flags(t) == 0 and np.isfinite(out).all() and np.isfinite(got).all()
    assert np.abs(out - want).max() <= 30 * 2.0 ** -22 * np.abs(h.v).max()
    assert (out[2] == 0).all()
    w, wt = ch.add_weights(h, share, [30 * 2.0 ** -22] * h.B)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_heads", [8, 16])
@pytest.mark.parametrize("down", [12, 24, 40])
def test_weights_beside_larger_ones(whole, fmt, q_heads, down):
    """One group in 16 has values 2^down times the others', in the upper half of the dims alone, and
    all scores are equal.  Each dim is held to its own sum: a weight p * sV keeps 2^-22 of itself or
    2^-37 of the largest of the step's eight groups (times that group's codes), all else is 2^-22 *
    30 of the sum of |p v| in the dim."""
    need_gpu()
    h = c4.History([4 * 400, 4 * 67], q_heads=q_heads, kv_heads=1, head_dim=64, fmt=fmt, seed=44)
    h.q[:] = 0
    big = np.arange(len(h.v)) // 4 % 16 == 3
    h.v[big, :, :32] = 0
    h.v[~big] *= np.float32(2.0 ** -down)
    h.set_cache()
    K, V = h.coded()
    rows = [np.arange(1600), np.arange(268)]
    t = c4.device(h, whole=whole)
    ch.fill_cache(h, t)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 512)
    out = _attend(t, ids, n).cpu().numpy().astype(np.float64)
    assert _flags(t) == 0
    for b, row in enumerate(rows):
        g = h.group_offset[b] + row[::4] // 4
        v = V[g, 0].reshape(-1, 64)
        x = h.v[h.token_offset[b] + row].reshape(-1, 4, 1, 64).transpose(0, 2, 1, 3)
        code, tile, s = c4.encode(x, fmt)
        s = s[:, 0].astype(np.float64)
        steps = np.concatenate([s, np.zeros(-len(s) % 8)]).reshape(-1, 8).max(axis=1)
        units = np.abs(code * np.repeat(tile, 4, axis=-1)[..., None, :])[:, 0]          # [groups, 4, d]
        floor = (np.repeat(steps, 8)[:len(s), None] * units.sum(axis=1)).sum(axis=0) / len(row)
        tol = 2.0 ** -22 * 30 * np.abs(v).mean(axis=0) + 2.0 ** -37 * floor
        err = np.abs(out[b] - v.mean(axis=0))
        assert (err <= tol).all(), (b, (err / tol).max())


@pytest.mark.parametrize("fmt", FORMATS)
def test_groups_that_are_not_finite_reach_only_what_attends_to_them(fmt):
    need_gpu()
    h = c4.History([400, 400], q_heads=4, kv_heads=2, head_dim=64, fmt=fmt, seed=19)
    h.k[40, 1, 5] = np.nan           # query 0, group 10, head 1
    h.v[400 + 44, 0, 3] = np.inf     # query 1, group 11, head 0
    h.set_cache()
    t = c4.device(h, whole=True)
    ch.fill_cache(h, t)
    out = _attend(t).cpu().numpy()
    assert np.isnan(out[0, 2:]).all() and np.isfinite(out[0, :2]).all()
    assert np.isnan(out[1, :2]).all() and np.isfinite(out[1, 2:]).all()
    ids, n = ch.rows_to_device([np.r_[0:40, 44:400], np.r_[0:44, 48:400]], 512)
    assert np.isfinite(_attend(t, ids, n).cpu().numpy()).all()
    assert _flags(t) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_flags_what_is_out_of_range(fmt):
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = c4.History([100, 203, 64, 40], q_heads=4, kv_heads=2, head_dim=64, fmt=fmt, seed=21)
    t = c4.device(h, budget=32, whole=True, weights=True)
    ch.fill_cache(h, t)
    good = _attend(t).clone()
    vis = t["visible"].clone()
    for bad in (-1, 204):
        t["visible"].copy_(vis)
        t["visible"][1] = bad
        before = t["weights"].clone()
        _attend(t, weights=True)
        assert _flags(t) == qsa.QSA_DEVERR_VISIBLE_RANGE
        assert (t["out"][1] == 0).all() and torch.equal(t["out"][[0, 2, 3]], good[[0, 2, 3]])
        lo = int(h.weight_offset[1])
        assert torch.equal(t["weights"][lo:lo + 51], before[lo:lo + 51])
    t["visible"].copy_(vis)
    # blocks outside the cache: zero rows, in a step of their own and beside others
    for gone in ([5], [0, 1, 2, 3], list(range(8, 16)), [15]):
        bm = t["block_map"].clone()
        K, V = h.coded()
        for i, g in enumerate(gone):
            t["block_map"][int(h.group_offset[2]) + g] = h.num_blocks + i if i % 2 else -1 - i
            K[h.group_offset[2] + g] = 0
            V[h.group_offset[2] + g] = 0
        ref, _, tol, _ = ch.attention(h, coded=(K, V))
        _close(h, _attend(t), ref, tol)
        assert _flags(t) == qsa.QSA_DEVERR_SLOT_RANGE
        t["block_map"].copy_(bm)
    # rows: counts out of range give zeros; a malformed group is a zero row, and the query adds no weight
    base = ch.some_rows(h, 20, 22)
    for b, change in enumerate(("neg", "long", "odd", "order")):
        ids, n = ch.rows_to_device([r.copy() for r in base], 32)
        if change == "neg":
            n[b] = -1
        elif change == "long":
            n[b] = 4 * 32 + 4
        elif change == "odd":
            ids[b, 9] += 1
        else:
            ids[b, :8] = torch.cat([ids[b, 4:8].clone(), ids[b, :4].clone()])
        before = t["weights"].clone()
        _attend(t, ids, n, weights=True)
        assert _flags(t) == qsa.QSA_DEVERR_ROW_RANGE, change
        lo, hi = int(h.weight_offset[b]), int(h.weight_offset[b]) + -(-int(h.visible[b]) // 4)
        assert torch.equal(t["weights"][lo:hi], before[lo:hi]), change
        if b < 2:
            assert (t["out"][b] == 0).all()
        if change == "order":  # the attention itself takes any order
            ref, _, tol, _ = ch.attention(h, base)
            _close(h, t["out"], ref, tol)


def test_a_captured_call_replays_on_new_inputs():
    """Coding, attention with weights and reading back captured once, replayed on other rows of the
    f32 cache, with eager calls on another workspace in between."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = c4.History([517, 66], q_heads=16, kv_heads=2, head_dim=128, fmt=c4.INT4, seed=23)
    t = c4.device(h, whole=True, weights=True)
    back = [torch.zeros_like(t["k_cache"]) for _ in range(2)]
    inp = qsa.QsaInputs(k_cache=back[0].data_ptr(), v_cache=back[1].data_ptr(), num_slots=h.num_slots,
                        slot_map=t["slot_map"].data_ptr(), slot_offset=t["token_offset"].data_ptr())

    def all_of_it():
        ch.fill_cache(h, t)
        _attend(t, weights=True)
        qsa.qsa_read_groups(t["dims"], inp, t["cache"], t["lo"], t["hi"], t["most"], t["ws"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        all_of_it()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        all_of_it()
    h2 = c4.History([517, 66], q_heads=16, kv_heads=2, head_dim=128, fmt=c4.INT4, seed=24)
    h2.slot_map, h2.block_map = h.slot_map, h.block_map
    h2.set_cache()
    for hh in (h2, h):
        t["k_cache"].copy_(torch.from_numpy(hh.k_cache))
        t["v_cache"].copy_(torch.from_numpy(hh.v_cache))
        t["q"].copy_(torch.from_numpy(hh.q))
        t["weights"].copy_(torch.from_numpy(hh.weights0))
        g.replay()
        ref, share, tol, rel = ch.attention(hh)
        _close(hh, t["out"], ref, tol)
        w, wt = ch.add_weights(hh, share, rel)
        assert (np.abs(t["weights"].cpu().numpy() - w) <= wt).all()
        K, _ = hh.coded()
        n = 517 // 4
        want = K[:n].astype(np.float32).transpose(0, 2, 1, 3).reshape(4 * n, 2, 128)
        assert np.array_equal(back[0].cpu().numpy()[h.slot_map[:4 * n]], want)
        t2 = c4.device(h, whole=True)
        ch.fill_cache(h, t2)
        _attend(t2)
        assert _flags(t2) == 0
    assert _flags(t) == 0


def test_caches_beyond_two_to_the_32():
    """Blocks whose codes start beyond byte 2^32: coded, attended to and read back as anywhere else."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = c4.History([70, 515], q_heads=16, kv_heads=2, head_dim=128, fmt=c4.E2M1, seed=61)
    t = c4.device(h, whole=True)
    high = 2 ** 32 // 1152 + 7
    codes = torch.zeros(high + h.num_blocks, 2, 576, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(high + h.num_blocks, 2, 2, device="cuda")
    t["block_map"] += high
    cache = qsa.QsaCodedCache.of(codes, scales, t["block_map"], t["group_offset"], h.fmt)
    qsa.qsa_code_groups(t["dims"], t["inputs"], cache, t["lo"], t["hi"], t["most"], t["ws"])
    qsa.qsa_attend_coded(t["dims"], t["inputs"], cache, None, None, t["out"], t["ws"])
    assert _flags(t) == 0
    assert (codes[:high] == 0).all()
    ref, _, tol, _ = ch.attention(h)
    _close(h, t["out"], ref, tol)
    tails = np.r_[68:70, 70 + 512:70 + 515]
    before = t["k_cache"].clone()
    qsa.qsa_read_groups(t["dims"], t["inputs"], cache, t["lo"], t["hi"], t["most"], t["ws"])
    assert _flags(t) == 0
    K, _ = h.coded()
    got = t["k_cache"].cpu().numpy()
    assert np.array_equal(got[h.slot_map[:68]], K[:17].astype(np.float32).transpose(0, 2, 1, 3).reshape(68, 2, 128))
    assert np.array_equal(got[h.slot_map[tails]], before.cpu().numpy()[h.slot_map[tails]])


def test_two_streams_at_once():
    torch = need_gpu()
    hs = [c4.History([9001, 515, 0, 4099], q_heads=16, kv_heads=2, head_dim=128, fmt=c4.E2M1, seed=71),
          c4.History([3, 2048, 7001], q_heads=16, kv_heads=1, head_dim=64, fmt=c4.INT4, seed=72)]
    ts = [c4.device(h, whole=True, weights=True) for h in hs]
    alone = []
    for h, t in zip(hs, ts):
        ch.fill_cache(h, t)
        _attend(t, weights=True)
        alone.append((t["out"].clone(), t["weights"].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    outs = [[], []]
    for _ in range(20):
        for i, (h, t, s) in enumerate(zip(hs, ts, streams)):
            with torch.cuda.stream(s):
                t["weights"].copy_(torch.from_numpy(h.weights0).pin_memory(), non_blocking=True)
                _attend(t, weights=True)
                outs[i].append((t["out"].clone(), t["weights"].clone()))
    torch.cuda.synchronize()
    for i in range(2):
        for out, w in outs[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(w, alone[i][1])
        assert _flags(ts[i]) == 0
