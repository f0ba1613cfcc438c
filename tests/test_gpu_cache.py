"""The coded cache, the attention over it and the eviction on the GPU, against
their plain forms in 64 bits (tests/cache_helpers.py)."""
import numpy as np
import pytest

import cache_helpers as ch
from gpu_helpers import ATTN_TOL, need_gpu

pytestmark = pytest.mark.gpu

LENGTHS = [0, 1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 67, 127, 128, 131, 509, 2048, 2051, 4096, 4099, 4101, 9001]
HEADS = [(1, 1, 64), (2, 2, 64), (8, 2, 64), (16, 2, 128), (16, 1, 128), (10, 2, 128), (12, 1, 64), (9, 1, 128), (24, 8, 128)]


def _ok(t):
    from top_group_sparse_gb300 import qsa
    st, flags = qsa.qsa_check_errors(t["ws"])
    assert st == 0, f"device error word {flags:#x}"


def _flags(t):
    from top_group_sparse_gb300 import qsa
    return qsa.qsa_check_errors(t["ws"])[1]


def _attend(t, ids=None, n_ids=None, weights=False, stream=None):
    from top_group_sparse_gb300 import qsa
    qsa.qsa_attend_coded(t["dims"], t["inputs"], t["cache"], ids, n_ids, t["out"], t["ws"],
                         weights=t["weights"] if weights else None,
                         weight_offset=t["weight_offset"] if weights else None, stream=stream)
    return t["out"]


def _close(h, got, ref, tol, standard=True):
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    for b in range(h.B):
        err = np.abs(got[b] - ref[b]).max()
        assert err <= tol[b], f"query {b} (T {h.visible[b]}): {err:.3e} > {tol[b]:.3e}"
        if standard:  # the library's bar for values drawn from N(0, 1)
            assert err <= ATTN_TOL * 6, f"query {b}"


# ---- coding ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("kv,d", [(1, 64), (3, 64), (2, 128), (8, 128)])
def test_codes_and_scales_equal_the_definition(fmt, kv, d):
    need_gpu()
    h = ch.History([0, 3, 4, 7, 64, 1029, 517], q_heads=kv, kv_heads=kv, head_dim=d, fmt=fmt, seed=3)
    h.k *= np.exp(3 * np.random.RandomState(1).randn(len(h.k), 1, 1)).astype(np.float32)
    h.k_cache[h.slot_map] = h.k
    t = ch.device(h)
    t["codes"].fill_(0x5a)
    t["scales"].fill_(-3.0)
    ch.fill_cache(h, t)
    _ok(t)
    K, V = ch.unpack(t["codes"].cpu().numpy(), d, fmt)
    s = t["scales"].cpu().numpy()
    done = np.zeros(h.num_blocks, bool)
    for b, T in enumerate(h.visible):
        n = int(T) // 4
        blk = h.block_map[h.group_offset[b]:h.group_offset[b] + n]
        done[blk] = True
        for src, got, i in ((h.k, K, 0), (h.v, V, 1)):
            x = src[h.token_offset[b]:h.token_offset[b] + 4 * n].reshape(n, 4, kv, d).transpose(0, 2, 1, 3)
            c, sc = ch.encode(x, fmt)
            assert np.array_equal(s[blk, :, i], sc)
            assert np.array_equal(got[blk], c)
    # blocks of no group are left as they were
    assert (t["codes"].cpu().numpy()[~done] == 0x5a).all() and (s[~done] == -3.0).all()


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_coding_of_extreme_groups(fmt, d):
    """Zero, tiny, subnormal, huge, infinite and NaN groups, each beside an ordinary one."""
    need_gpu()
    vals = [0.0, 1e-45, 1e-38, 5e-36, 6e-36, 1e-30, 3.0e38, np.inf, -np.inf, np.nan, 1.0]
    h = ch.History([4 * len(vals)], q_heads=2, kv_heads=2, head_dim=d, fmt=fmt, seed=5)
    for i, v in enumerate(vals):
        if v == 0 or abs(v) < 1e-20:
            h.k[4 * i:4 * i + 4] = (np.random.RandomState(i).rand(4, 2, d) * v).astype(np.float32)
        h.k[4 * i + i % 4, 0, (7 * i) % d] = v     # head 0 only
        h.v[4 * i + 3, 1, (5 * i) % d] = v
    h.k_cache[h.slot_map], h.v_cache[h.slot_map] = h.k, h.v
    t = ch.device(h)
    ch.fill_cache(h, t)
    _ok(t)
    K, V = ch.unpack(t["codes"].cpu().numpy(), d, fmt)
    s = t["scales"].cpu().numpy()
    blk = h.block_map[:len(vals)]
    for src, got, j in ((h.k, K, 0), (h.v, V, 1)):
        x = src.reshape(len(vals), 4, 2, d).transpose(0, 2, 1, 3)
        c, sc = ch.encode(x, fmt)
        assert np.array_equal(s[blk, :, j], sc, equal_nan=True)
        assert np.array_equal(got[blk], c)


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("log2_scale", [-120, -89, -40, 0, 3, 100])
def test_codes_next_to_the_borders_between_codes(fmt, log2_scale):
    """Values at, and one or two units beside, the middle of two codes: the rounded
    quotient decides, and a quotient that is off by one unit shows."""
    need_gpu()
    r = np.random.RandomState(8)
    n, d = 400, 64
    h = ch.History([4 * n], q_heads=1, kv_heads=1, head_dim=d, fmt=fmt, seed=9)
    grid = np.unique(np.abs(ch.e4m3_table()[:0x7f])) if fmt == ch.E4M3 else np.arange(128.0)
    mid = (grid[1:] + grid[:-1]) / 2
    for a in (h.k, h.v):
        amax = (2.0 ** log2_scale * (1 + r.rand(n))).astype(np.float32)
        s = amax * (np.float32(1) / np.float32(ch.QMAX[fmt]))
        x = (mid[r.randint(0, len(mid), (n, 4 * d))] * s[:, None].astype(np.float64)).astype(np.float32)
        x = (x.view(np.int32) + r.randint(-2, 3, x.shape).astype(np.int32)).view(np.float32) * r.choice([-1, 1], x.shape).astype(np.float32)
        x = np.clip(x, -amax[:, None], amax[:, None])
        x[np.arange(n), r.randint(0, 4 * d, n)] = amax
        a[:] = x.reshape(4 * n, 1, d)
    h.k_cache[h.slot_map], h.v_cache[h.slot_map] = h.k, h.v
    t = ch.device(h)
    ch.fill_cache(h, t)
    _ok(t)
    K, V = ch.unpack(t["codes"].cpu().numpy(), d, fmt)
    s = t["scales"].cpu().numpy()
    blk = h.block_map[:n]
    for src, got, j in ((h.k, K, 0), (h.v, V, 1)):
        c, sc = ch.encode(src.reshape(n, 4, 1, d).transpose(0, 2, 1, 3), fmt)
        assert np.array_equal(s[blk, :, j], sc)
        assert np.array_equal(got[blk], c)


def test_coding_flags_and_skips_what_is_out_of_range():
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = ch.History([64, 64, 64], q_heads=2, kv_heads=2, head_dim=64, fmt=ch.E4M3, seed=6)
    t = ch.device(h)
    for lo, hi, most in (([-1, 0, 0], [1, 0, 0], 1), ([0, 5, 0], [0, 4, 0], 1), ([0, 0, 16], [0, 0, 17], 1), ([0, 0, 0], [0, 2, 0], 1)):
        t["codes"].fill_(9)
        qsa.qsa_code_groups(t["dims"], t["inputs"], t["cache"], torch.tensor(lo, dtype=torch.int32, device="cuda"),
                            torch.tensor(hi, dtype=torch.int32, device="cuda"), most, t["ws"])
        assert _flags(t) == qsa.QSA_DEVERR_VISIBLE_RANGE
        assert (t["codes"] == 9).all()
    # a block outside the cache is skipped, a slot outside it codes zeros; the others are coded
    bm, sl = t["block_map"].clone(), t["slot_map"].clone()
    t["block_map"][3] = h.num_blocks
    t["block_map"][4] = -1
    t["slot_map"][8] = h.num_slots
    t["slot_map"][9] = -7
    t["codes"].zero_()
    ch.fill_cache(h, t)
    assert _flags(t) == qsa.QSA_DEVERR_SLOT_RANGE
    K, _ = ch.unpack(t["codes"].cpu().numpy(), 64, h.fmt)
    for g in range(48):
        if g in (3, 4):
            assert (K[int(bm[g])] == 0).all()
            continue
        x = h.k[4 * g:4 * g + 4].copy()
        if g == 2:
            x[:2] = 0
        assert np.array_equal(K[int(bm[g])], ch.encode(x.transpose(1, 0, 2), h.fmt)[0]), g
    t["block_map"].copy_(bm)
    t["slot_map"].copy_(sl)
    # the same block named by two queries of one history
    h = ch.History([40, 40], q_heads=2, kv_heads=2, head_dim=64, fmt=ch.E4M3, seed=7, shared=True)
    t = ch.device(h)
    both = torch.tensor([10, 10], dtype=torch.int32, device="cuda")
    qsa.qsa_code_groups(t["dims"], t["inputs"], t["cache"], both - 10, both, 10, t["ws"])
    _ok(t)
    K, _ = ch.unpack(t["codes"].cpu().numpy(), 64, h.fmt)
    assert np.array_equal(K[h.block_map[:10]], ch.encode(h.k.reshape(10, 4, 2, 64).transpose(0, 2, 1, 3), h.fmt)[0])


# ---- attention ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("q_heads,kv,d", HEADS)
def test_attention_over_whole_histories(fmt, q_heads, kv, d):
    need_gpu()
    h = ch.History(LENGTHS, q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=11)
    t = ch.device(h, whole=True, weights=True)
    ch.fill_cache(h, t)
    ref, share, tol, rel = ch.attention(h)
    _close(h, _attend(t), ref, tol)
    _ok(t)
    first = t["out"].clone()
    # with weights: the same output, and the shares added
    _attend(t, weights=True)
    _ok(t)
    assert (t["out"] == first).all()
    w, wt = ch.add_weights(h, share, rel)
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()
    assert abs((got - h.weights0).sum() - q_heads * np.count_nonzero(h.visible)) < 1e-3 * q_heads


@pytest.mark.parametrize("fmt,q_heads", [(ch.E4M3, 3), (ch.INT8, 12)])
def test_attention_over_long_histories(fmt, q_heads):
    """Rows on both sides of each change of the run length, whose runs take several
    segments, beside short ones."""
    need_gpu()
    h = ch.History([4 * 4097 + 1, 5, 4 * 4096, 4 * 65537 + 2, 4 * 131073 + 3], q_heads=q_heads, kv_heads=1, head_dim=64, fmt=fmt,
                   seed=27)
    t = ch.device(h, whole=True, weights=True)
    ch.fill_cache(h, t)
    ref, share, tol, rel = ch.attention(h)
    # (more runs per slice and more steps per warp than the bound of shorter rows counts: 512/8 + 128 additions)
    vmax = max(float(np.abs(h.v).max()), 1.0) * 1.1
    _close(h, _attend(t, weights=True), ref, tol + vmax * 192 * 2.0 ** -24)
    _ok(t)
    w, wt = ch.add_weights(h, share, [r + 192 * 2.0 ** -24 for r in rel])
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()


@pytest.mark.parametrize("budget", [512, 32, 5, 1])
@pytest.mark.parametrize("fmt,q_heads,kv,d", [(ch.E4M3, 16, 2, 128), (ch.INT8, 8, 2, 64), (ch.INT8, 16, 1, 128), (ch.E4M3, 3, 3, 64)])
def test_attention_over_selected_rows(budget, fmt, q_heads, kv, d):
    need_gpu()
    h = ch.History([0, 1, 3, 4, 6, 70, 128, 131, 2051, 9002, 4097], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=12)
    rows = ch.some_rows(h, budget, 13)
    t = ch.device(h, budget=budget, weights=True)
    ch.fill_cache(h, t)
    ids, n = ch.rows_to_device(rows, budget)
    ref, share, tol, rel = ch.attention(h, rows)
    _close(h, _attend(t, ids, n), ref, tol)
    first = t["out"].clone()
    _attend(t, ids, n, weights=True)
    _ok(t)
    assert (t["out"] == first).all()
    w, wt = ch.add_weights(h, share, rel)
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()


@pytest.mark.parametrize("whole", [True, False])
def test_weights_of_a_shared_history_are_added_in_batch_order(whole):
    torch = need_gpu()
    vis = [989 + i for i in range(39)]  # up to 1,027: 256 groups and a tail of 3
    h = ch.History(vis, q_heads=8, kv_heads=2, head_dim=64, fmt=ch.INT8, seed=14, shared=True)
    t = ch.device(h, budget=64, whole=whole, weights=True)
    ch.fill_cache(h, t)
    rows = None if whole else ch.some_rows(h, 64, 15)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 64)
    ref, share, tol, rel = ch.attention(h, rows)
    _close(h, _attend(t, ids, n, weights=True), ref, tol)
    _ok(t)
    w, wt = ch.add_weights(h, share, rel)
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()
    again = t["weights"].clone()
    for _ in range(3):
        t["weights"].copy_(torch.from_numpy(h.weights0))
        _attend(t, ids, n, weights=True)
        assert torch.equal(t["weights"], again)


@pytest.mark.parametrize("whole", [True, False])
def test_weights_of_several_shared_histories_in_one_batch(whole):
    """600 queries: five histories dealt out in turn (sharers far apart, beyond one
    block of 256), and some queries with accumulators of their own among them."""
    torch = need_gpu()
    r = np.random.RandomState(24)
    B = 600
    h = ch.History([int(t) for t in r.randint(1, 90, B)], q_heads=2, kv_heads=1, head_dim=64, fmt=ch.E4M3, seed=25)
    room = 24  # groups per accumulator row
    own = r.rand(B) < 0.1
    pick = np.where(own, 5 + np.arange(B), np.arange(B) % 5)
    pick[300:560][~own[300:560]] = 2
    h.weight_offset = (pick * room).astype(np.int64)
    h.n_weights = (5 + B) * room
    h.weights0 = r.rand(h.n_weights).astype(np.float32)
    rows = None if whole else ch.some_rows(h, 9, 26)
    t = ch.device(h, budget=9, whole=whole, weights=True)
    ch.fill_cache(h, t)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 9)
    _, share, _, rel = ch.attention(h, rows)
    _attend(t, ids, n, weights=True)
    _ok(t)
    w, wt = ch.add_weights(h, share, rel)
    got = t["weights"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= wt).all(), np.abs(got - w).max()
    again = t["weights"].clone()
    t["weights"].copy_(torch.from_numpy(h.weights0))
    _attend(t, ids, n, weights=True)
    assert torch.equal(t["weights"], again)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("sharers", [2, 3, 8, 9, 12, 530])
def test_a_shared_sum_does_not_depend_on_the_rest_of_the_batch(whole, sharers):
    """Queries that share accumulators add the same bits alone and among queries of
    other histories (each with accumulators of its own, or shared by two)."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    r = np.random.RandomState(27)
    B = 3 * sharers
    mine = np.sort(r.permutation(B)[:sharers])
    h = ch.History([int(t) for t in r.randint(1, 400, B)], q_heads=4, kv_heads=1, head_dim=64, fmt=ch.E4M3, seed=28)
    room = 100
    pick = 1 + np.arange(B) // 2
    pick[mine] = 0
    h.weight_offset = (pick * room).astype(np.int64)
    h.n_weights = (2 + B) * room
    h.weights0 = r.rand(h.n_weights).astype(np.float32)
    budget = 40
    t = ch.device(h, budget=budget, whole=whole, weights=True, max_visible=400)
    ch.fill_cache(h, t)
    rows = None if whole else ch.some_rows(h, budget, 29)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, budget)
    _, share, _, rel = ch.attention(h, rows)
    _attend(t, ids, n, weights=True)
    _ok(t)
    w, wt = ch.add_weights(h, share, rel)
    assert (np.abs(t["weights"].cpu().numpy() - w) <= wt).all()
    among = t["weights"][:room].clone()
    sel = torch.from_numpy(mine).cuda()
    one = {k: t[k][sel].contiguous() for k in ("visible", "q", "token_offset", "group_offset", "weight_offset")}
    dims = qsa.make_dims(sharers, 8, 64, 4, 1, 64, budget_groups=budget, max_visible=400, scale=h.scale)
    ws = torch.zeros(qsa.qsa_coded_workspace_size(dims, whole, True), dtype=torch.uint8, device="cuda")
    inp = qsa.QsaInputs(visible=one["visible"].data_ptr(), q=one["q"].data_ptr(), k_cache=t["k_cache"].data_ptr(),
                        v_cache=t["v_cache"].data_ptr(), num_slots=h.num_slots, slot_map=t["slot_map"].data_ptr(),
                        slot_offset=one["token_offset"].data_ptr())
    cache = qsa.QsaCodedCache.of(t["codes"], t["scales"], t["block_map"], one["group_offset"], h.fmt)
    alone = torch.from_numpy(h.weights0).cuda()
    out = torch.empty(sharers, 4, 64, device="cuda")
    some = (None, None) if whole else (ids[sel].contiguous(), n[sel].contiguous())
    qsa.qsa_attend_coded(dims, inp, cache, *some, out, ws, weights=alone, weight_offset=one["weight_offset"])
    assert torch.equal(alone[:room], among)


@pytest.mark.parametrize("whole", [True, False])
def test_weights_of_many_shared_histories(whole):
    """300 histories of two queries each, interleaved: more units of work than CTAs."""
    torch = need_gpu()
    r = np.random.RandomState(30)
    B, room = 600, 260
    h = ch.History([int(t) for t in r.randint(800, 1030, B)], q_heads=2, kv_heads=1, head_dim=64, fmt=ch.INT8, seed=31)
    h.weight_offset = (np.arange(B) % 300 * room).astype(np.int64)
    h.n_weights = 300 * room
    h.weights0 = r.rand(h.n_weights).astype(np.float32)
    t = ch.device(h, budget=20, whole=whole, weights=True)
    ch.fill_cache(h, t)
    rows = None if whole else ch.some_rows(h, 20, 32)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 20)
    _, share, _, rel = ch.attention(h, rows)
    _attend(t, ids, n, weights=True)
    _ok(t)
    w, wt = ch.add_weights(h, share, rel)
    assert (np.abs(t["weights"].cpu().numpy() - w) <= wt).all()
    again = t["weights"].clone()
    t["weights"].copy_(torch.from_numpy(h.weights0))
    _attend(t, ids, n, weights=True)
    assert torch.equal(t["weights"], again)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("vis,q_heads,kv", [([3, 2, 1, 3, 0], 2, 1), ([1029, 1027, 1025], 80, 8), ([67, 0, 3], 130, 65)])
def test_weights_of_raw_tails_alone_and_of_many_heads(vis, q_heads, kv, whole, shared):
    """Histories without a complete group, and more heads than a block of threads has statistics for."""
    need_gpu()
    h = ch.History(vis, q_heads=q_heads, kv_heads=kv, head_dim=64, fmt=ch.E4M3, seed=33, shared=shared)
    t = ch.device(h, budget=7, whole=whole, weights=True)
    ch.fill_cache(h, t)
    rows = None if whole else ch.some_rows(h, 7, 34)
    ids, n = (None, None) if whole else ch.rows_to_device(rows, 7)
    ref, share, tol, rel = ch.attention(h, rows)
    _close(h, _attend(t, ids, n, weights=True), ref, tol)
    _ok(t)
    # (a share sums up to 130 heads, not the 16 that the helper counts)
    w, wt = ch.add_weights(h, share, [x + q_heads * 2.0 ** -24 for x in rel])
    assert (np.abs(t["weights"].cpu().numpy() - w) <= wt).all()


def test_the_longest_history():
    """QSA_MAX_VISIBLE tokens less one beside a short history: 2^24 groups that name 61
    blocks in turn, so that the result is a sum over 61 blocks with their counts.
    The tokens of a run of 32,768 groups enter a warp's sums in 2,048 additions and
    512 runs are merged by 64: each leaves half a step."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    nb, T = 61, 2 ** 26 - 1
    G = T // 4
    h = ch.History([4 * nb + 3, 4 * nb + 3], q_heads=2, kv_heads=1, head_dim=64, fmt=ch.E4M3, seed=35, shared=True)
    t = ch.device(h, whole=True)
    ch.fill_cache(h, t)
    visible = torch.tensor([T, 4 * nb + 3], dtype=torch.int32, device="cuda")
    block_map = torch.empty(G + nb, dtype=torch.int32, device="cuda")
    block_map[:G] = t["block_map"][torch.arange(G, device="cuda") % nb]
    block_map[G:] = t["block_map"]
    block_offset = torch.tensor([0, G], dtype=torch.int64, device="cuda")
    slot_map = torch.full((T + 4 * nb + 3,), -7, dtype=torch.int32, device="cuda")  # read for the raw tails alone
    slot_map[T - 3:T] = t["slot_map"][4 * nb:]
    slot_map[T + 4 * nb:] = t["slot_map"][4 * nb:]
    slot_offset = torch.tensor([0, T], dtype=torch.int64, device="cuda")
    weights = torch.zeros(G + 1 + nb + 1, device="cuda")
    weight_offset = torch.tensor([0, G + 1], dtype=torch.int64, device="cuda")
    dims = qsa.make_dims(2, 8, 64, 2, 1, 64, max_visible=2 ** 26, scale=h.scale)
    ws = torch.zeros(qsa.qsa_coded_workspace_size(dims, True, True), dtype=torch.uint8, device="cuda")
    inp = qsa.QsaInputs(visible=visible.data_ptr(), q=t["q"].data_ptr(), k_cache=t["k_cache"].data_ptr(),
                        v_cache=t["v_cache"].data_ptr(), num_slots=h.num_slots, slot_map=slot_map.data_ptr(),
                        slot_offset=slot_offset.data_ptr())
    cache = qsa.QsaCodedCache.of(t["codes"], t["scales"], block_map, block_offset, h.fmt)
    out = torch.full((2, 2, 64), float("nan"), device="cuda")
    qsa.qsa_attend_coded(dims, inp, cache, None, None, out, ws, weights=weights, weight_offset=weight_offset)
    assert qsa.qsa_check_errors(ws)[1] == 0
    K, V = h.coded()
    K = np.concatenate([K[:nb, 0].reshape(-1, 64), h.k[4 * nb:4 * nb + 3, 0]]).astype(np.float64)
    V = np.concatenate([V[:nb, 0].reshape(-1, 64), h.v[4 * nb:4 * nb + 3, 0]]).astype(np.float64)
    got, w = out.cpu().numpy(), weights.cpu().numpy().astype(np.float64)
    rel = 2.0 ** -24 * (2 * (2048 + 64 + 16) + 4 * 30) + 2.0 ** -22 * 14 * 16
    for b, groups in ((0, G), (1, nb)):
        count = np.bincount(np.arange(groups) % nb, minlength=nb).astype(np.float64)
        share = np.zeros(nb + 1)
        for hd in range(2):
            p = np.exp((h.q[b, hd].astype(np.float64) @ K.T) * h.scale)
            n = np.concatenate([np.repeat(count, 4), np.ones(3)])
            Z = (p * n).sum()
            assert np.abs((np.abs(h.q[b, hd]) @ np.abs(K).T) * h.scale).max() < 16
            assert np.abs(got[b, hd] - (p * n) @ V / Z).max() <= rel * np.abs(V).max()
            share += np.concatenate([p[:4 * nb].reshape(nb, 4).sum(1), [p[4 * nb:].sum()]]) / Z
        off = 0 if b == 0 else G + 1
        want = np.concatenate([share[np.arange(groups) % nb], share[nb:]])
        assert (np.abs(w[off:off + groups + 1] - want) <= rel * want).all()
    # and its eviction, down to half
    keep = G // 2
    kept = torch.full((2, keep), -1, dtype=torch.int32, device="cuda")
    n_kept = torch.zeros(2, dtype=torch.int32, device="cuda")
    qsa.qsa_evict_select(dims, visible, weights, weight_offset, keep, 4, 1000, kept, n_kept, ws)
    assert n_kept.tolist() == [keep, nb] and torch.equal(kept[1, :nb].cpu(), torch.arange(nb, dtype=torch.int32))
    ref = ch.evict([T], w, [0], keep, 4, 1000)[0]
    assert np.array_equal(kept[0].cpu().numpy(), ref)


def test_an_output_does_not_depend_on_the_batch_or_the_workspace():
    """Each query alone, in a workspace made for its own length, gives the bits it
    gives in the batch, call after call."""
    torch = need_gpu()
    h = ch.History([4101, 77, 9001, 0, 640], q_heads=16, kv_heads=2, head_dim=128, fmt=ch.E4M3, seed=16)
    t = ch.device(h, whole=True)
    ch.fill_cache(h, t)
    out = _attend(t).clone()
    assert torch.equal(_attend(t), out)
    from top_group_sparse_gb300 import qsa
    for b in range(h.B):
        dims = qsa.make_dims(1, 8, 64, 16, 2, 128, max_visible=int(h.visible[b]) + 1000 * b, scale=h.scale)
        ws = torch.zeros(qsa.qsa_coded_workspace_size(dims, True), dtype=torch.uint8, device="cuda")
        inp = qsa.QsaInputs(visible=t["visible"][b:].data_ptr(), q=t["q"][b:].data_ptr(), k_cache=t["k_cache"].data_ptr(),
                            v_cache=t["v_cache"].data_ptr(), num_slots=h.num_slots, slot_map=t["slot_map"].data_ptr(),
                            slot_offset=t["token_offset"][b:].data_ptr())
        cache = qsa.QsaCodedCache.of(t["codes"], t["scales"], t["block_map"], t["group_offset"][b:], h.fmt)
        one = torch.full((1, 16, 128), float("nan"), device="cuda")
        qsa.qsa_attend_coded(dims, inp, cache, None, None, one, ws)
        assert torch.equal(one[0], out[b]), b


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
@pytest.mark.parametrize("q_heads,kv,d", HEADS)
def test_rows_of_one_run_give_the_same_bits_as_among_longer_ones(q_heads, kv, d, fmt):
    """Calls whose rows are all short enough for one run: against 64 bits, and bit for
    bit against the same rows in a call that allows longer ones."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    vis = [0, 1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 66, 131, 252, 255, 256]
    h = ch.History(vis, q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=36)
    for rows in (None, ch.some_rows(h, 13, 37)):
        budget = 13 if rows else 512
        t = ch.device(h, budget=budget, whole=rows is None, max_visible=259)
        ch.fill_cache(h, t)
        ids, n = ch.rows_to_device(rows, budget) if rows else (None, None)
        ref, _, tol, _ = ch.attention(h, rows)
        _close(h, _attend(t, ids, n), ref, tol)
        _ok(t)
        short = t["out"].clone()
        if rows:  # budgets of more than one run
            budget = 80
            ids, n = ch.rows_to_device(rows, budget)
        dims = qsa.make_dims(h.B, 8, 64, q_heads, kv, d, budget_groups=budget, max_visible=9001, scale=h.scale)
        ws = torch.zeros(qsa.qsa_coded_workspace_size(dims, rows is None), dtype=torch.uint8, device="cuda")
        out = torch.full_like(short, float("nan"))
        qsa.qsa_attend_coded(dims, t["inputs"], t["cache"], ids, n, out, ws)
        assert torch.equal(out, short)


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8])
def test_wide_ranges_of_scales_and_scores(fmt):
    """Scores spread over hundreds (one token takes all the weight), queries and
    groups whose sizes differ by 2^40, zero queries."""
    need_gpu()
    h = ch.History([2000, 2000, 333, 1200], q_heads=8, kv_heads=2, head_dim=128, fmt=fmt, seed=17)
    r = np.random.RandomState(18)
    h.q[0] *= 60
    h.q[2] = 0
    h.q[3] *= 2.0 ** -20
    for x in (h.k, h.v):
        x[h.token_offset[3]:] *= 2.0 ** 20
    h.v[:2000] *= np.repeat(2.0 ** r.randint(-20, 20, 500), 4)[:, None, None].astype(np.float32)
    h.k_cache[h.slot_map], h.v_cache[h.slot_map] = h.k, h.v
    t = ch.device(h, whole=True)
    ch.fill_cache(h, t)
    ref, _, tol, _ = ch.attention(h)
    _close(h, _attend(t), ref, tol, standard=False)
    _ok(t)


def test_groups_that_are_not_finite_reach_only_what_attends_to_them():
    need_gpu()
    h = ch.History([400, 400], q_heads=4, kv_heads=2, head_dim=64, fmt=ch.INT8, seed=19)
    h.k[40, 1, 5] = np.nan           # query 0, group 10, head 1
    h.v[400 + 44, 0, 3] = np.inf     # query 1, group 11, head 0
    h.k_cache[h.slot_map], h.v_cache[h.slot_map] = h.k, h.v
    t = ch.device(h, whole=True)
    ch.fill_cache(h, t)
    out = _attend(t).cpu().numpy()
    assert np.isnan(out[0, 2:]).all() and np.isfinite(out[0, :2]).all()
    assert np.isnan(out[1, :2]).all() and np.isfinite(out[1, 2:]).all()
    # rows without those groups
    rows = [np.r_[0:40, 44:400], np.r_[0:44, 48:400]]
    ids, n = ch.rows_to_device(rows, 512)
    out = _attend(t, ids, n).cpu().numpy()
    assert np.isfinite(out).all()
    _ok(t)
    # what the f32 cache holds in slots that no tail names is not read
    h = ch.History([402, 7], q_heads=4, kv_heads=2, head_dim=64, fmt=ch.INT8, seed=20)
    t = ch.device(h, whole=True)
    ch.fill_cache(h, t)
    tails = np.concatenate([h.slot_map[400:402], h.slot_map[402 + 4:402 + 7]])
    other = np.setdiff1d(np.arange(h.num_slots), tails)
    t["k_cache"][other] = float("nan")
    t["v_cache"][other] = float("inf")
    ref, _, tol, _ = ch.attention(h)
    _close(h, _attend(t), ref, tol)


def test_attention_flags_what_is_out_of_range():
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = ch.History([100, 203, 64, 40], q_heads=4, kv_heads=2, head_dim=64, fmt=ch.E4M3, seed=21)
    t = ch.device(h, budget=32, whole=True, weights=True)
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
        assert torch.equal(t["weights"][lo:lo + 51], before[lo:lo + 51])  # adds no weight
        assert (t["weights"][:25] > before[:25]).all()
    t["visible"].copy_(vis)
    # blocks and slots outside their caches: zero rows
    bm = t["block_map"].clone()
    t["block_map"][int(h.group_offset[2]) + 5] = h.num_blocks
    K, V = h.coded()
    K[h.group_offset[2] + 5] = 0
    V[h.group_offset[2] + 5] = 0
    sl = t["slot_map"].clone()
    t["slot_map"][int(h.token_offset[1]) + 202] = -1
    kk, vv = h.k.copy(), h.v.copy()
    h.k[h.token_offset[1] + 202] = 0
    h.v[h.token_offset[1] + 202] = 0
    ref, _, tol, _ = ch.attention(h, coded=(K, V))
    _close(h, _attend(t), ref, tol)
    assert _flags(t) == qsa.QSA_DEVERR_SLOT_RANGE
    h.k, h.v = kk, vv
    t["block_map"].copy_(bm)
    t["slot_map"].copy_(sl)
    # rows: counts out of range give zeros; a malformed group is a zero row, and the query adds no weight
    base = ch.some_rows(h, 20, 22)
    for b, change in enumerate(("neg", "long", "odd", "order")):
        rows = [r.copy() for r in base]
        ids, n = ch.rows_to_device(rows, 32)
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
        others = [o for o in range(4) if o != b]
        for o in others:
            lo, hi = int(h.weight_offset[o]), int(h.weight_offset[o]) + -(-int(h.visible[o]) // 4)
            assert not torch.equal(t["weights"][lo:hi], before[lo:hi])
        if b < 2:
            assert (t["out"][b] == 0).all()
        if change == "order":  # the attention itself takes any order
            ref, _, tol, _ = ch.attention(h, base)
            _close(h, t["out"], ref, tol)


def test_a_captured_call_replays_on_new_inputs_and_another_stream():
    """Coding and attention with weights captured once, replayed on other rows of the
    f32 cache, with eager calls on another workspace in between."""
    torch = need_gpu()
    h = ch.History([517, 66], q_heads=16, kv_heads=2, head_dim=128, fmt=ch.INT8, seed=23)
    t = ch.device(h, whole=True, weights=True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ch.fill_cache(h, t)
        _attend(t, weights=True)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ch.fill_cache(h, t)
        _attend(t, weights=True)
    h2 = ch.History([517, 66], q_heads=16, kv_heads=2, head_dim=128, fmt=ch.INT8, seed=24)
    h2.slot_map, h2.block_map = h.slot_map, h.block_map
    h2.k_cache[h.slot_map], h2.v_cache[h.slot_map] = h2.k, h2.v
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
        t2 = ch.device(h, whole=True)
        ch.fill_cache(h, t2)
        _attend(t2)
        _ok(t2)
    _ok(t)


def test_device_batch_runs_the_coded_cache():
    """DeviceBatch: coding, the whole path and the observation of whole histories,
    independent ones and a shared one."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    from top_group_sparse_gb300 import workloads as wl
    for vis, history in (([300, 2053, 0, 7], "independent"), ([997, 998, 1001, 1003], "shared")):
        w = wl.make_workload("coded", vis, idx_heads=4, idx_dim=32, q_heads=8, kv_heads=2, head_dim=64, seed=51, slots="paged16",
                             history=history, budget=33)
        db = qsa.DeviceBatch(w)
        db.make_coded_cache(qsa.QSA_CODE_INT8)
        db.code_all()
        db.decode_coded(weigh=True)
        assert qsa.qsa_check_errors(db.coded_ws)[1] == 0
        h = ch.History(vis, q_heads=8, kv_heads=2, head_dim=64, fmt=ch.INT8, seed=52, shared=history == "shared")
        h.q, h.k, h.v = w.q, w.k_cache[w.slot_map], w.v_cache[w.slot_map]
        h.weights0 = np.zeros(max(h.n_weights, 1), np.float32)
        assert np.array_equal(db.weight_offset.cpu().numpy(), h.weight_offset)
        rows = [db.ids[b, :int(db.n_ids[b])].cpu().numpy() for b in range(4)]
        ref, share, tol, rel = ch.attention(h, rows)
        _close(h, db.out, ref, tol)
        wt, at = ch.add_weights(h, share, rel)
        assert (np.abs(db.weights.cpu().numpy() - wt) <= at).all()
        db.attend_coded()
        _close(h, db.out, ref, tol)
        db.weights.zero_()
        db.attend_coded(whole=True, weigh=True)
        ref, share, tol, rel = ch.attention(h)
        _close(h, db.out, ref, tol)
        wt, at = ch.add_weights(h, share, rel)
        assert (np.abs(db.weights.cpu().numpy() - wt) <= at).all()
        assert qsa.qsa_check_errors(db.coded_ws)[1] == 0


def test_device_batch_codes_on_the_stream_it_is_given():
    """Calls one after the other on a side stream that is far behind, with other work taking
    and filling memory meanwhile: each still finds its own ranges.  Ranges of another
    length than the batch are refused."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    from top_group_sparse_gb300 import workloads as wl
    w = wl.make_workload("coded", [301, 2053, 1000, 7], idx_heads=4, idx_dim=32, q_heads=8, kv_heads=2, head_dim=64, seed=53,
                         slots="paged16", budget=33)
    db = qsa.DeviceBatch(w)
    db.make_coded_cache()
    db.code_all()
    torch.cuda.synchronize()
    codes, scales = db.codes.clone(), db.scales.clone()
    db.codes.zero_()
    db.scales.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    G = np.array(w.visible) // 4
    cuts = [G * i // 5 for i in range(6)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    for i in range(5):
        db.code(cuts[i], cuts[i + 1], stream=side.cuda_stream if i % 2 else side)
        junk = [torch.full((4,), -1, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    assert len(junk) == 64 and qsa.qsa_check_errors(db.coded_ws)[1] == 0
    assert torch.equal(db.codes, codes) and torch.equal(db.scales, scales)
    for bad in ([0, 0, 0], [[0, 0, 0, 0]], 0):
        with pytest.raises(ValueError):
            db.code(bad, bad)


def test_caches_beyond_two_to_the_31():
    """Blocks whose codes start beyond byte 2^31 and slots whose rows start beyond
    element 2^31: coded, and attended to, as anywhere else."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    h = ch.History([70, 515], q_heads=16, kv_heads=2, head_dim=128, fmt=ch.INT8, seed=61)
    t = ch.device(h, whole=True)
    high_slot, high_block = 2 ** 31 // 256 + 5, 2 ** 31 // 2048 + 7
    num_slots, num_blocks = high_slot + h.num_slots, high_block + h.num_blocks
    k = torch.zeros(num_slots, 2, 128, device="cuda")
    v = torch.zeros(num_slots, 2, 128, device="cuda")
    k[high_slot:].copy_(t["k_cache"])
    v[high_slot:].copy_(t["v_cache"])
    codes = torch.zeros(num_blocks, 2, 1024, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(num_blocks, 2, 2, device="cuda")
    t["slot_map"] += high_slot
    t["block_map"] += high_block
    inp = qsa.QsaInputs(visible=t["visible"].data_ptr(), q=t["q"].data_ptr(), k_cache=k.data_ptr(), v_cache=v.data_ptr(),
                        num_slots=num_slots, slot_map=t["slot_map"].data_ptr(), slot_offset=t["token_offset"].data_ptr())
    cache = qsa.QsaCodedCache.of(codes, scales, t["block_map"], t["group_offset"], h.fmt)
    qsa.qsa_code_groups(t["dims"], inp, cache, t["lo"], t["hi"], t["most"], t["ws"])
    qsa.qsa_attend_coded(t["dims"], inp, cache, None, None, t["out"], t["ws"])
    _ok(t)
    assert (codes[:high_block] == 0).all()
    ref, _, tol, _ = ch.attention(h)
    _close(h, t["out"], ref, tol)


def test_two_streams_at_once():
    """Two batches on two streams, each with a workspace of its own, many times over:
    both give what they give alone."""
    torch = need_gpu()
    hs = [ch.History([9001, 515, 0, 4099], q_heads=16, kv_heads=2, head_dim=128, fmt=ch.E4M3, seed=71),
          ch.History([3, 2048, 7001], q_heads=8, kv_heads=8, head_dim=64, fmt=ch.INT8, seed=72)]
    ts = [ch.device(h, whole=True, weights=True) for h in hs]
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
        _ok(ts[i])
