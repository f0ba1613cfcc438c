"""The binding of qsa_append_tokens refuses tensors that the call would read past, before it is made (no GPU: the
library is replaced)."""
import types

import pytest

from top_group_sparse_gb300 import qsa

torch = pytest.importorskip("torch")
B, DIMS = 3, dict(idx_heads=4, idx_dim=32, q_heads=4, kv_heads=2, head_dim=64, max_visible=100)


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(qsa, "load", lambda: types.SimpleNamespace(qsa_append_tokens=lambda *a: made.append(a) or 0))
    return made


def _tensors(**kw):
    t = dict(q=torch.zeros(B, 256), k=torch.zeros(B, 2, 64), v=torch.zeros(B, 128), q_idx=torch.zeros(B, 4, 32),
             idx_key=torch.zeros(B, 32), positions=torch.zeros(B, dtype=torch.int32), freq=torch.zeros(32),
             idx_freq=torch.zeros(16), q_norm=torch.ones(64), k_norm=torch.ones(64), q_idx_norm=torch.ones(32),
             idx_key_norm=torch.ones(32))
    t.update(kw)
    return {n: x for n, x in t.items() if x is not None}


def _call(batch=B, through_the_batch=False, **kw):
    t = _tensors(**kw)
    dims, inputs, ws = qsa.make_dims(batch, **DIMS), qsa.QsaInputs(), torch.zeros(256, dtype=torch.uint8)
    tokens = qsa.QsaNewTokens.of(**t)
    if through_the_batch:
        db = object.__new__(qsa.DeviceBatch)
        db.dims, db.inputs, db.ws = dims, inputs, ws
        return db.append(tokens, 0)
    return qsa.qsa_append_tokens(dims, inputs, tokens, ws, 0)


SHORT = [dict(q=torch.zeros(B - 1, 256)), dict(q=torch.zeros(1, 256)), dict(k=torch.zeros(B - 1, 2, 64)),
         dict(v=torch.zeros(B - 1, 128)), dict(q_idx=torch.zeros(B - 1, 128)), dict(idx_key=torch.zeros(2, 32)),
         dict(q=torch.zeros(B, 512)[:, :192]), dict(k=torch.zeros(B, 1, 128)[:, :, :64]), dict(v=torch.zeros(B, 512)[:, :64]),
         dict(q_idx=torch.zeros(B, 512)[:, :96]), dict(idx_key=torch.zeros(B, 512)[:, :16]),
         dict(q_norm=torch.ones(32)), dict(k_norm=torch.ones(60)), dict(q_idx_norm=torch.ones(16)), dict(idx_key_norm=torch.ones(1)),
         dict(positions=torch.zeros(B - 1, dtype=torch.int32)), dict(positions=torch.zeros(1, B - 1, dtype=torch.int32)),
         dict(positions=torch.zeros(2, B - 1, dtype=torch.int32), freq=torch.zeros(2, 32), idx_freq=torch.zeros(2, 16)),
         dict(positions=torch.zeros(2, B + 1, dtype=torch.int32), freq=torch.zeros(2, 32), idx_freq=torch.zeros(2, 16)),
         dict(positions=torch.zeros(B - 1, dtype=torch.int32), freq=None),
         dict(positions=torch.zeros(B - 1, dtype=torch.int32), idx_freq=None)]


@pytest.mark.parametrize("short", SHORT)
@pytest.mark.parametrize("through_the_batch", [False, True])
def test_short_tensors_are_refused(calls, short, through_the_batch):
    with pytest.raises(ValueError):
        _call(through_the_batch=through_the_batch, **short)
    assert not calls


LONG = [dict(), dict(q=torch.zeros(B + 2, 256)), dict(q=torch.zeros(B, 512)[:, :256]), dict(k=torch.zeros(B, 160)),
        dict(q_norm=torch.ones(128)), dict(positions=torch.zeros(B + 5, dtype=torch.int32)), dict(positions=torch.zeros(1, B + 5, dtype=torch.int32)),
        dict(positions=torch.zeros(1, dtype=torch.int32), freq=None, idx_freq=None),   # nothing turns, nothing is read
        dict(positions=torch.zeros(1, dtype=torch.int32), idx_freq=None, q=None, k=None, q_norm=None, k_norm=None)]


@pytest.mark.parametrize("more", LONG)
def test_what_is_long_enough_passes(calls, more):
    assert _call(**more) == 0 and len(calls) == 1


def test_one_row_for_a_batch_of_several_and_structures_of_pointers(calls):
    assert _call(batch=1) == 0 and _call(batch=0) == 0
    with pytest.raises(ValueError):
        _call(batch=B + 1)
    t = qsa.QsaNewTokens(q=qsa.QsaProjection(1 << 20, 256, None), type=0, axes=1)   # made of pointers: it knows no sizes
    assert qsa.qsa_append_tokens(qsa.make_dims(5, **DIMS), qsa.QsaInputs(), t, torch.zeros(256, dtype=torch.uint8), 0) == 0
    assert len(calls) == 3


def test_pointers_put_in_the_place_of_a_tensor_are_taken_as_they_are(calls):
    dims, ws = qsa.make_dims(2 * B, **DIMS), torch.zeros(256, dtype=torch.uint8)
    t = qsa.QsaNewTokens.of(q=torch.zeros(B, 256), q_norm=torch.ones(32), positions=torch.zeros(2, B, dtype=torch.int32), freq=torch.zeros(2, 32))
    for change in (lambda: setattr(t.q, "rows", 1 << 20), lambda: setattr(t.q, "norm", 1 << 21), lambda: setattr(t, "positions", 1 << 22)):
        with pytest.raises(ValueError):
            qsa.qsa_append_tokens(dims, qsa.QsaInputs(), t, ws, 0)
        change()
    assert qsa.qsa_append_tokens(dims, qsa.QsaInputs(), t, ws, 0) == 0 and len(calls) == 1


def test_dims_that_change_between_calls(calls):
    dims, ws = qsa.make_dims(B, **DIMS), torch.zeros(256, dtype=torch.uint8)
    t = qsa.QsaNewTokens.of(**_tensors())
    for batch, head_dim, q_heads, fits in ((B, 64, 4, True), (B, 64, 4, True), (B + 1, 64, 4, False), (B, 128, 2, False), (B, 64, 5, False),
                                           (1, 64, 4, True), (B + 1, 64, 4, False), (B, 64, 4, True)):
        dims.batch, dims.head_dim, dims.q_heads = batch, head_dim, q_heads
        before = len(calls)
        if fits:
            assert qsa.qsa_append_tokens(dims, qsa.QsaInputs(), t, ws, 0) == 0
        else:
            with pytest.raises(ValueError):
                qsa.qsa_append_tokens(dims, qsa.QsaInputs(), t, ws, 0)
        assert len(calls) == before + fits
