"""DeviceBatch.code_all and read_back take every complete group of every history, by the queries' lengths as they are
at the call and not as they were when the cache was made."""
import numpy as np
import pytest

from top_group_sparse_gb300 import qsa
from top_group_sparse_gb300 import workloads as wl

torch = pytest.importorskip("torch")


def _workload(visible, history="shared"):
    return wl.make_workload("moved", visible, idx_heads=4, idx_dim=32, q_heads=8, kv_heads=2, head_dim=64, seed=61, history=history,
                            slots="paged16", budget=33)


@pytest.mark.parametrize("made,now,want", [
    ([9, 13, 21], [9, 13, 21], [0, 0, 5]), ([9, 13, 21], [21, 9, 13], [5, 0, 0]), ([9, 13, 21], [8, 20, 3], [0, 5, 0]),
    ([9, 13, 21], [0, 0, 0], [0, 0, 0]), ([21, 21, 21], [16, 20, 20], [0, 5, 0]), ([5], [4], [1]), ([], [], [])])
def test_the_ends_of_a_shared_history(monkeypatch, made, now, want):
    from top_group_sparse_gb300 import build
    build.build()
    db = qsa.DeviceBatch(_workload(made), device="cpu")
    db.make_coded_cache(qsa.QSA_CODE_INT4)
    db.visible.copy_(torch.tensor(now, dtype=torch.int32))
    coded = []
    monkeypatch.setattr(db, "code", lambda lo, hi, stream: coded.append((lo.tolist(), hi.tolist())))
    db.code_all()
    assert coded == [([0] * len(made), want)]


def test_the_ends_of_histories_of_their_own():
    from top_group_sparse_gb300 import build
    build.build()
    db = qsa.DeviceBatch(_workload([21, 0, 9, 40], "independent"), device="cpu")
    db.make_coded_cache()
    for now, want in (([21, 0, 9, 40], [5, 0, 2, 10]), ([3, 0, 8, 40], [0, 0, 2, 10]), ([21, 0, -1, 40], [5, 0, -1, 10])):
        db.visible.copy_(torch.tensor(now, dtype=torch.int32))
        assert db._whole_histories().tolist() == want and db._whole_histories().dtype == np.int32


def test_groups_without_a_block_are_refused(monkeypatch):
    """A history that has grown past the blocks it was given: its next entries of the block map are another
    history's, or past the end."""
    from top_group_sparse_gb300 import build
    build.build()
    calls = []
    for name in ("qsa_code_groups", "qsa_read_groups"):
        monkeypatch.setattr(qsa, name, lambda *a: calls.append(a[3:6]))
    monkeypatch.setattr(qsa, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: __import__("contextlib").nullcontext())
    db = qsa.DeviceBatch(_workload([40, 40, 40], "independent"), device="cpu")
    db.visible.copy_(torch.tensor([20, 11, 40], dtype=torch.int32))
    db.make_coded_cache()
    for grown, bad in (([24, 11, 40], 0), ([20, 12, 40], 1), ([23, 40, 8], 1)):
        db.visible.copy_(torch.tensor(grown, dtype=torch.int32))
        ge = np.array(grown) // 4
        for call in (db.code_all, db.read_back, lambda: db.code(ge - 1, ge)):
            with pytest.raises(ValueError, match=f"query {bad}: groups up to {ge[bad]} "):
                call()
    assert not calls
    db.visible.copy_(torch.tensor([23, 8, 40], dtype=torch.int32))
    db.code_all()
    db.read_back()
    db.code([0, 9, 10], [5, 9, 10])          # (an empty range anywhere)
    assert [(lo.tolist(), hi.tolist(), n) for lo, hi, n in calls] == [([0, 0, 0], [5, 2, 10], 10)] * 2 + [([0, 9, 10], [5, 9, 10], 5)]
    db.visible.copy_(torch.tensor([40, 40, 40], dtype=torch.int32))
    db.coded = qsa.QsaCodedCache.of(db.codes, db.scales, db.block_map, db.block_offset, 0)  # the caller's own: not looked into
    db.code_all()
    assert calls[-1][2] == 10


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [qsa.QSA_CODE_E4M3, qsa.QSA_CODE_INT4])
def test_a_history_whose_longest_query_is_another_one(fmt):
    from gpu_helpers import need_gpu
    need_gpu()
    w = _workload([300, 517, 77])
    db = qsa.DeviceBatch(w)
    db.make_coded_cache(fmt)
    db.visible.copy_(torch.tensor([516, 3, 131], dtype=torch.int32))
    db.code_all()
    assert db.check_errors() == (0, 0)
    assert (db.scales[:129] > 0).all()       # every group has been coded
    slots = torch.from_numpy(w.slot_map[:516].astype(np.int64)).cuda()
    was = db.k_cache[slots].clone()
    db.k_cache.fill_(-9)
    db.v_cache.fill_(-9)
    db.read_back()
    assert db.check_errors() == (0, 0)
    got = db.k_cache[slots]
    assert (got != -9).all() and (db.v_cache[slots] != -9).all()
    assert (got - was).abs().max() <= (0.25 if fmt == qsa.QSA_CODE_INT4 else 0.07) * was.abs().max()
