"""qsa_append_tokens on the GPU against its plain form in 64 bits (tests/rows_helpers.py), and
the new calls run together as a serving step runs them."""
import numpy as np
import pytest

import cache4_helpers as c4
import cache_helpers as ch
import rows_helpers as rh
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

SHAPES = [  # q heads, KV heads, d, indexer heads, d_I
    (16, 2, 128, 8, 64), (1, 1, 64, 4, 32), (8, 8, 64, 8, 32), (10, 2, 128, 4, 64), (3, 1, 64, 5, 64), (64, 8, 128, 8, 64),
    (40, 40, 64, 33, 32)]


def _append(t, stream=None):
    from top_group_sparse_gb300 import qsa
    qsa.qsa_append_tokens(t["dims"], t["inputs"], t["tokens"], t["ws"], stream)


def _run(b, type_name="f32", **kw):
    from top_group_sparse_gb300 import qsa
    t = b.on_device(type_name, **kw)
    _append(t)
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    b.check(t, type_name)
    return t


def _batch(visible, shape, **kw):
    nq, kv, d, ih, di = shape
    kw.setdefault("seed", 3)
    return rh.Batch(visible, q_heads=nq, kv_heads=kv, head_dim=d, idx_heads=ih, idx_dim=di, **kw)


@pytest.mark.parametrize("type_name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pairing", [rh.HALVES, rh.NEIGHBOURS])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_of_every_shape_and_type(shape, pairing, type_name):
    need_gpu()
    _run(_batch([5, 1, 0, 33, 2], shape, pairing=pairing, axes=2, pad=8), type_name)


@pytest.mark.parametrize("pairing", [rh.HALVES, rh.NEIGHBOURS])
@pytest.mark.parametrize("dims,idx_dims", [(0, 0), (8, 8), (16, 24), (24, 32), (56, 0), (64, 40), (72, 56), (120, 64), (128, 48)])
def test_every_kind_of_partial_rotation(dims, idx_dims, pairing):
    """Partners an odd and an even number of quads away, in the same lane and in others; dims that do not turn."""
    need_gpu()
    for norms in (True, False):
        _run(_batch([7, 3, 1], (6, 2, 128, 5, 64), dims=dims, idx_dims=idx_dims, pairing=pairing,
                    idx_pairing=1 - pairing, norms=norms), "bf16")


@pytest.mark.parametrize("given", [("q",), ("k",), ("v",), ("q_idx",), ("idx_key",), ("k", "v"), ("q", "idx_key"), ("v", "q_idx"),
                                   ("q", "k", "v"), ("q_idx", "idx_key")])
def test_projections_that_are_not_given_write_nothing(given):
    need_gpu()
    b = _batch([5, 0, 9, 2], (6, 2, 64, 4, 32), given=given)
    _run(b)
    # .. and what no given projection needs may be NULL
    from top_group_sparse_gb300 import qsa
    t = b.on_device()
    need = {"visible"} | {"q": {"q"}, "k": {"k_cache"}, "v": {"v_cache"}, "q_idx": {"q_idx"}, "idx_key": {"idx_keys", "key_offset"}}[given[0]]
    for g in given[1:]:
        need |= {"q": {"q"}, "k": {"k_cache"}, "v": {"v_cache"}, "q_idx": {"q_idx"}, "idx_key": {"idx_keys", "key_offset"}}[g]
    if {"k", "v"} & set(given):
        need |= {"slot_map", "slot_offset"}
    inp = t["inputs"]
    t["inputs"] = qsa.QsaInputs(num_slots=inp.num_slots, **{n: getattr(inp, n) for n in need})
    _append(t)
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    b.check(t)


def test_nothing_is_rotated_without_positions():
    need_gpu()
    from top_group_sparse_gb300 import qsa
    b = _batch([5, 2], (6, 2, 64, 4, 32), dims=0, idx_dims=0)
    t = b.on_device()
    assert t["tokens"].turn.dims == 0
    t["tokens"].positions = None
    _append(t)
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    b.check(t)


@pytest.mark.parametrize("type_name", ["f32", "bf16"])
@pytest.mark.parametrize("B", [1, 31, 607, 2500])
def test_batches_that_take_several_tokens_at_a_time(B, type_name):
    """Consecutive positions of one history; several tokens per CTA, and several rounds of them."""
    need_gpu()
    n = 4 if B > 600 else 16
    _run(_batch([100 + i for i in range(B)], (n, 2, 64, 4, 32), shared=True, axes=3, dims=16, idx_dims=16), type_name)


def test_the_largest_batch():
    """65,535 tokens, one row of one head each: bit for bit what the same tokens give 500 at a time."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    b = _batch(np.arange(1, 65536), (2, 1, 64, 4, 32), shared=True, given=("q", "k", "idx_key"), dims=64, idx_dims=0, far=1 << 30)
    t = b.on_device("bf16")
    _append(t)
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    whole = [t[n].clone() for n in ("q", "k_cache", "idx_keys")]
    assert (whole[0] != -9).all() and (whole[2] != -9).all()
    for n in ("q", "k_cache", "idx_keys"):
        t[n].fill_(-9)
    for at in range(0, b.B, 5000):
        m = min(500, b.B - at)
        dims = qsa.make_dims(m, 4, 32, 2, 1, 64, max_visible=65535)
        inp = qsa.QsaInputs(num_slots=b.num_slots, visible=t["visible"][at:].data_ptr(), q=t["q"][at:].data_ptr(),
                            k_cache=t["k_cache"].data_ptr(), slot_map=t["slot_map"].data_ptr(), slot_offset=t["offset"].data_ptr(),
                            v_cache=t["v_cache"].data_ptr(), idx_keys=t["idx_keys"].data_ptr(), key_offset=t["offset"].data_ptr())
        tok = qsa.QsaNewTokens.of(**{k: t["fused"][at:at + m, b.slice[k]] for k in b.given},
                                  positions=t["positions"][:, at:at + m].contiguous(), freq=t["freq"]["turn"], eps=b.eps,
                                  **{k + "_norm": t["norm"][k] for k in b.given})
        qsa.qsa_append_tokens(dims, inp, tok, t["ws"])
        torch.cuda.synchronize()
        assert torch.equal(t["q"][at:at + m], whole[0][at:at + m]) and torch.equal(t["idx_keys"][at:at + m], whole[2][at:at + m])
        slot = t["slot_map"][at:at + m].long()
        assert torch.equal(t["k_cache"][slot], whole[1][slot])
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)


@pytest.mark.parametrize("align", [16, 32])
def test_outputs_on_sixteen_bytes_and_on_thirty_two(align):
    need_gpu()
    _run(_batch([5, 2, 8], (6, 2, 128, 4, 64)), "bf16", align=align)


def test_far_negative_and_extreme_positions():
    """The angle keeps its fraction of a turn whatever the position."""
    need_gpu()
    from top_group_sparse_gb300 import qsa
    b = _batch([3] * 8, (4, 2, 64, 4, 32), norms=False, axes=4)
    b.positions[0] = [0, 1, -1, 2 ** 26, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321]
    b.positions[1] = [0, -7, 2 ** 31 - 1, 5, -2 ** 31, 2 ** 31 - 1, 11, 2 ** 24 + 1]
    b.turn["turn"][2] = -b.turn["turn"][0][::-1]                              # negative, and all axes at once
    b.turn["turn"][3] = np.array([65535.9, 1e-30, 1e-42, 0.5] * 8, np.float32)  # the largest, and next to none
    t = b.on_device()
    _append(t)
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    b.check(t)


def test_frequencies_out_of_range_make_their_pairs_nan():
    need_gpu()
    b = _batch([3, 4], (4, 2, 64, 4, 32), norms=False)
    bad = [np.inf, -np.inf, np.nan, 65536.0, -1e30]
    b.turn["turn"][0, :5] = bad
    t = b.on_device()
    _append(t)
    q = t["q"].cpu().numpy()
    assert np.isnan(q[..., :5]).all() and np.isnan(q[..., 32:37]).all()
    b.turn["turn"][0, :5] = 0
    y, tol = b.expected("f32")["q"]
    ok = np.r_[5:32, 37:64]
    assert (np.abs(q[..., ok] - y[..., ok]) <= tol[..., ok]).all()


def test_values_that_are_not_finite_stay_in_their_heads():
    """An infinity or a NaN in one head leaves the others as they are; without a norm it reaches its pair alone,
    and a dim that does not turn is copied."""
    need_gpu()
    b = _batch([3, 4], (4, 2, 64, 4, 32), norms=False, dims=32)
    b.fused[0, 64 + 40] = np.inf        # q head 1, a dim that does not turn
    b.fused[1, 2 * 64 + 3] = np.nan     # q head 2, paired with dim 19
    t = b.on_device()
    _append(t)
    q = t["q"].cpu().numpy()
    assert q[0, 1, 40] == np.inf and np.isfinite(np.delete(q[0].ravel(), 64 + 40)).all()
    assert np.isnan(q[1, 2, [3, 19]]).all() and np.isfinite(np.delete(q[1].ravel(), [131, 147])).all()
    b = _batch([3, 4], (4, 2, 64, 4, 32), dims=32)
    b.fused[0, 64 + 40] = np.nan
    t = b.on_device()
    _append(t)
    q = t["q"].cpu().numpy()
    assert np.isnan(q[0, 1]).all() and np.isfinite(q[0, [0, 2, 3]]).all() and np.isfinite(q[1]).all()


@pytest.mark.parametrize("size", [1e-18, 1e18])
def test_norms_of_small_and_large_heads(size):
    """Squares near both ends of binary32; eps decides what is far below its root."""
    need_gpu()
    _run(_batch([3, 4, 9], (4, 2, 64, 4, 32), eps=0.0 if size > 1 else 1e-30, values=lambda r, s: (size * r.randn(*s)).astype(np.float32)))
    _run(_batch([3, 4, 9], (4, 2, 64, 4, 32), eps=1e-5, values=lambda r, s: np.zeros(s, np.float32)))


def test_device_errors_leave_the_caches_alone():
    need_gpu()
    from top_group_sparse_gb300 import qsa
    b = _batch([5, 2, 8, 1], (6, 2, 64, 4, 32))
    for bad in (-1, 9):
        t = b.on_device()
        t["visible"][1] = bad
        _append(t)
        assert qsa.qsa_check_errors(t["ws"])[1] == qsa.QSA_DEVERR_VISIBLE_RANGE
        assert (t["q"][1] == 0).all() and (t["q_idx"][1] == 0).all()
        t["q"][1] = t["q_idx"][1] = -9
        keep, b.visible = b.visible, b.visible.copy()
        b.visible[1] = 0
        b.check(t)
        b.visible = keep
    t = b.on_device()
    row = int(b.offset[2]) + 7
    for bad in (-1, b.num_slots):
        t["slot_map"][row] = bad
        t["k_cache"].fill_(-9)
        t["v_cache"].fill_(-9)
        _append(t)
        assert qsa.qsa_check_errors(t["ws"])[1] == qsa.QSA_DEVERR_SLOT_RANGE
        got = t["k_cache"].cpu().numpy()
        assert (got[b.slot_map[row]] == -9).all() and (got[b.slot_map[[4, 6, 15]]] != -9).all()
        y, tol = b.expected("f32")["q"]
        assert (np.abs(t["q"].cpu().numpy() - y) <= tol).all()


def test_rows_that_are_the_queries_themselves():
    """f32 rows of q and q_idx normalised and rotated in place, many tokens at once."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    b = _batch([10 + i for i in range(1500)], (4, 1, 64, 4, 32), shared=True, given=("q", "q_idx"), dims=16, idx_dims=8)
    t = b.on_device()
    t["q"].copy_(t["fused"][:, b.slice["q"]].view_as(t["q"]))
    t["q_idx"].copy_(t["fused"][:, b.slice["q_idx"]].view_as(t["q_idx"]))
    t["tokens"] = qsa.QsaNewTokens.of(q=t["q"], q_idx=t["q_idx"], positions=t["positions"], freq=t["freq"]["turn"],
                                      idx_freq=t["freq"]["turn_idx"], eps=b.eps, q_norm=t["norm"]["q"], q_idx_norm=t["norm"]["q_idx"])
    _append(t)
    torch.cuda.synchronize()
    b.check(t)


@pytest.mark.parametrize("shape,tokens,type_name", [((1, 1, 64, 4, 32), 20011, "bf16"), ((32, 8, 128, 8, 64), 4099, "f16"),
                                                    ((16, 2, 128, 8, 64), 6007, "f32"), ((8, 2, 64, 4, 64), 9001, "bf16")])
def test_more_tokens_than_are_taken_at_once(shape, tokens, type_name):
    """Several rounds of every CTA, with queries that bring nothing and ends inside a round."""
    need_gpu()
    visible = np.random.default_rng(5).integers(0, 4, tokens)
    _run(_batch(visible, shape, axes=2, dims=shape[2], idx_dims=24), type_name)


def test_a_captured_call_replays_on_another_stream():
    torch = need_gpu()
    b = _batch([5, 2, 8, 1], (16, 2, 128, 8, 64), axes=3)
    t = b.on_device("bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _append(t)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _append(t)
    b2 = _batch([5, 2, 8, 1], (16, 2, 128, 8, 64), axes=3, seed=4)
    b2.slot_map, b2.norm, b2.turn = b.slot_map, b.norm, b.turn
    t["fused"].copy_(torch.from_numpy(b2.fused))
    t["positions"].copy_(torch.from_numpy(b2.positions))
    for n in ("q", "q_idx", "k_cache", "v_cache", "idx_keys"):
        t[n].fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    b2.check(t, "bf16")


def test_a_token_gives_the_same_bits_in_every_batch():
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    b = _batch([5, 2, 8, 1, 0, 40] * 300, (16, 2, 128, 8, 64), axes=2)
    t = _run(b, "f16")
    for at in (0, 1, 5, 777):
        dims = qsa.make_dims(1, 8, 64, 16, 2, 128, max_visible=40)
        one = torch.full((1, 16, 128), -9.0, device="cuda")
        k = torch.full_like(t["k_cache"], -9.0)
        inp = qsa.QsaInputs(num_slots=b.num_slots, visible=t["visible"][at:].data_ptr(), q=one.data_ptr(), k_cache=k.data_ptr(),
                            slot_map=t["slot_map"].data_ptr(), slot_offset=t["offset"][at:].data_ptr())
        tok = qsa.QsaNewTokens.of(q=t["fused"][at:at + 1, b.slice["q"]], k=t["fused"][at:at + 1, b.slice["k"]],
                                  positions=t["positions"][:, at:at + 1].contiguous(), freq=t["freq"]["turn"], eps=b.eps,
                                  q_norm=t["norm"]["q"], k_norm=t["norm"]["k"])
        qsa.qsa_append_tokens(dims, inp, tok, t["ws"])
        torch.cuda.synchronize()
        assert torch.equal(one[0], t["q"][at])
        slot = int(b.slot_map[b.offset[at] + b.visible[at] - 1])
        assert torch.equal(k[slot], t["k_cache"][slot])


@pytest.mark.parametrize("fmt", [c4.E2M1, c4.INT4])
def test_a_serving_loop_over_a_cache_in_four_bits(fmt):
    """Twelve decode steps of two sequences from projections alone: append, pool and code what completes,
    decode over the 4-bit cache; then the histories read back.  Against the same steps in 64 bits over
    the codes of the plain form."""
    torch = need_gpu()
    import oracle
    from top_group_sparse_gb300 import qsa
    from top_group_sparse_gb300 import workloads as wl
    start, steps, budget = [61, 1030], 12, 24
    w = wl.make_workload("loop", [t + steps for t in start], idx_heads=4, idx_dim=32, q_heads=8, kv_heads=2, head_dim=64, seed=5,
                         slots="paged16", budget=budget)
    db = qsa.DeviceBatch(w)
    db.make_pooled_cache()
    db.make_coded_cache(fmt)
    vis = np.array(start, np.int32)
    db.visible.copy_(torch.from_numpy(vis))
    db.pool(np.zeros(2, np.int32), vis // 4)
    db.code(np.zeros(2, np.int32), vis // 4)
    r = np.random.RandomState(6)
    freq = (10000.0 ** (-np.arange(0, 64, 2) / 64.0)).astype(np.float32)[None]
    idx_freq = (10000.0 ** (-np.arange(0, 16, 2) / 16.0)).astype(np.float32)[None]
    norm = (1 + 0.1 * r.randn(64)).astype(np.float32)
    dev = {n: torch.from_numpy(a).cuda() for n, a in (("freq", freq), ("idx_freq", idx_freq), ("norm", norm))}
    for step in range(steps):
        vis += 1
        db.visible.copy_(torch.from_numpy(vis))
        x = {"q": r.randn(2, 8 * 64), "k": r.randn(2, 2 * 64), "v": r.randn(2, 2 * 64), "q_idx": r.randn(2, 4 * 32), "idx_key": r.randn(2, 32)}
        x = {n: torch.from_numpy(a).cuda().to(torch.bfloat16) for n, a in x.items()}
        pos = torch.from_numpy(vis - 1).cuda()
        tok = qsa.QsaNewTokens.of(**x, positions=pos, freq=dev["freq"], idx_freq=dev["idx_freq"], q_norm=dev["norm"],
                                  k_norm=dev["norm"], eps=1e-6)
        db.append(tok)
        # the token's own rows, from the definition
        ang = rh.angles((vis - 1)[None], freq)
        y = x["k"].float().cpu().numpy().astype(np.float64).reshape(2, 2, 64)
        y = y / np.sqrt((y ** 2).mean(axis=2, keepdims=True) + 1e-6) * norm
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y = np.concatenate([y[..., :32] * c - y[..., 32:] * s, y[..., :32] * s + y[..., 32:] * c], axis=2)
        slot = [int(w.slot_map[w.slot_offset[b] + vis[b] - 1]) for b in range(2)]
        # (rows_helpers: 3 * 2^-21 of |y_i| + |y_k|, each at most sqrt(2) of the largest turned one)
        assert np.abs(db.k_cache.cpu().numpy()[slot] - y).max() < 2.0 ** -18 * np.abs(y).max()
        done = np.where(vis % 4 == 0, 1, 0).astype(np.int32)
        if done.any():
            db.pool(vis // 4 - done, vis // 4)
            db.code(vis // 4 - done, vis // 4)
        qsa.qsa_decode_coded(db.dims, db.inputs, db.coded, db.ids, db.n_ids, db.out, db.coded_ws, pooled=db.pooled,
                             pool_offset=db.pool_offset)
        assert db.check_errors() == (0, 0)
        if step % 5 != 1:
            continue
        # rows: the oracle's, over the arrays as they stand; outputs: attention over the plain form's codes
        w.visible[:] = vis
        w.q_idx[:], w.q[:] = db.q_idx.cpu().numpy(), db.q.cpu().numpy()
        w.idx_keys[:], w.k_cache[:], w.v_cache[:] = (a.cpu().numpy() for a in (db.idx_keys, db.k_cache, db.v_cache))
        ref = oracle.decode(w)
        for b in range(2):
            n = int(ref["n_ids"][b])
            assert int(db.n_ids[b]) == n and np.array_equal(db.ids[b, :n].cpu().numpy(), ref["ids"][b, :n])
        h = c4.History(vis, q_heads=8, kv_heads=2, head_dim=64, fmt=fmt, seed=7)
        for b in range(2):
            sl = w.slot_map[w.slot_offset[b]:w.slot_offset[b] + vis[b]]
            h.k[h.token_offset[b]:h.token_offset[b] + vis[b]], h.v[h.token_offset[b]:h.token_offset[b] + vis[b]] = w.k_cache[sl], w.v_cache[sl]
        h.q = w.q.copy()
        rows = [ref["ids"][b, :int(ref["n_ids"][b])] for b in range(2)]
        want, _, tol, _ = ch.attention(h, rows)
        got = db.out.cpu().numpy().astype(np.float64)
        for b in range(2):
            assert np.abs(got[b] - want[b]).max() <= tol[b]
    # and the histories back in f32
    before = db.k_cache.clone()
    db.read_back()
    assert db.check_errors() == (0, 0)
    K, _ = h.coded() if step % 5 == 1 else (None, None)
    for b in range(2):
        n = int(vis[b]) // 4
        sl = torch.from_numpy(w.slot_map[w.slot_offset[b]:w.slot_offset[b] + vis[b]].astype(np.int64)).cuda()
        src = before[sl[:4 * n]].cpu().numpy().reshape(n, 4, 2, 64).transpose(0, 2, 1, 3)
        code, tile, s = c4.encode(src, fmt)
        want = (code * np.repeat(tile, 4, axis=-1)[..., None, :] * s.astype(np.float64)[..., None, None]).astype(np.float32)
        assert np.array_equal(db.k_cache[sl[:4 * n]].cpu().numpy(), want.transpose(0, 2, 1, 3).reshape(4 * n, 2, 64))
        assert torch.equal(db.k_cache[sl[4 * n:]], before[sl[4 * n:]])
