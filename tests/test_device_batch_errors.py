"""DeviceBatch.check_errors covers every workspace that the batch's calls use."""
import pytest

from top_group_sparse_gb300 import qsa


def test_both_workspaces_are_read_and_their_flags_joined(monkeypatch):
    words = {"plain": 0, "coded": 0}
    read = []

    def fake(ws, stream=None):
        read.append((ws, stream))
        flags, words[ws] = words[ws], 0
        return (qsa.QSA_ERR_DEVICE_FAULT if flags else qsa.QSA_OK), flags

    monkeypatch.setattr(qsa, "qsa_check_errors", fake)
    db = object.__new__(qsa.DeviceBatch)
    db.ws, db.coded_ws = "plain", None
    words["plain"] = 2
    assert db.check_errors() == (qsa.QSA_ERR_DEVICE_FAULT, 2) and db.check_errors() == (0, 0)
    assert {w for w, _ in read} == {"plain"}
    db.coded_ws = "coded"
    words.update(coded=4)
    assert db.check_errors(7) == (qsa.QSA_ERR_DEVICE_FAULT, 4) and read[-1] == ("coded", 7)
    words.update(plain=1, coded=4)
    assert db.check_errors() == (qsa.QSA_ERR_DEVICE_FAULT, 5) and db.check_errors() == (0, 0)


@pytest.mark.gpu
def test_an_error_of_a_coded_call_is_seen():
    from gpu_helpers import need_gpu
    need_gpu()
    from top_group_sparse_gb300 import workloads as wl
    w = wl.make_workload("coded", [300, 77], idx_heads=4, idx_dim=32, q_heads=8, kv_heads=2, head_dim=64, seed=61,
                         slots="paged16", budget=33)
    db = qsa.DeviceBatch(w)
    db.make_coded_cache()
    db.code_all()
    db.decode_coded(weigh=True)
    db.attend_coded(whole=True)
    assert db.check_errors() == (0, 0)
    db.block_map[5] = db.codes.shape[0]  # outside the cache: taken as zero rows, and flagged
    db.attend_coded(whole=True)
    assert db.check_errors() == (qsa.QSA_ERR_DEVICE_FAULT, qsa.QSA_DEVERR_SLOT_RANGE)
    assert db.check_errors() == (0, 0)
