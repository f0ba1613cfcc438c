"""include/qsa_rows.h and the 4-bit formats of include/qsa_cache.h on the host: every declared
symbol is exported, the structures are laid out as in C, and every refusal that the host can make
is made before anything is enqueued (no GPU here: a call that enqueued something would fail)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import cache4_helpers as c4
from top_group_sparse_gb300 import build as qbuild
from top_group_sparse_gb300 import qsa

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
INC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(qsa.__file__))), "include")
CALLS = ["qsa_append_tokens", "qsa_read_groups"]
F = 1 << 20  # aligned, not null, never dereferenced


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def _dims(**kw):
    base = dict(batch=2, idx_heads=8, idx_dim=64, q_heads=16, kv_heads=2, head_dim=128, budget_groups=512, max_visible=4096)
    base.update(kw)
    return qsa.make_dims(**base)


def _inputs(**kw):
    base = dict(q_idx=F, idx_keys=F, key_offset=F, visible=F, q=F, k_cache=F, v_cache=F, num_slots=100, slot_map=F,
                slot_offset=F)
    base.update(kw)
    return qsa.QsaInputs(**base)


def _cache(**kw):
    base = dict(codes=F, scales=F, num_blocks=100, block_map=F, block_offset=F, format=4)
    base.update(kw)
    return qsa.QsaCodedCache(**base)


def _tokens(**kw):
    base = dict(q=qsa.QsaProjection(F, 2048, F), k=qsa.QsaProjection(F, 256, F), v=qsa.QsaProjection(F, 256, None),
                q_idx=qsa.QsaProjection(F, 512, F), idx_key=qsa.QsaProjection(F, 64, F), type=1, axes=1, positions=F,
                turn=qsa.QsaRotation(F, 128, 0), turn_idx=qsa.QsaRotation(F, 64, 1), eps=1e-6)
    base.update(kw)
    return qsa.QsaNewTokens(**base)


def test_every_declared_symbol_is_exported(lib):
    assert qsa.exported_symbols(os.path.join(INC, "qsa_rows.h")) == CALLS
    for n in CALLS:
        assert hasattr(lib, n) and n in qsa.__all__
    for n in qsa.__all__:
        assert hasattr(qsa, n)


_C = r"""
#include <stddef.h>
#include <stdio.h>
#include "qsa_rows.h"

int main(void)
{
    static qsa_new_tokens t;
    printf("%zu %zu %zu %zu %zu %zu %zu %zu %d %d\n", sizeof(qsa_projection), sizeof(qsa_rotation), sizeof t,
           offsetof(qsa_new_tokens, type), offsetof(qsa_new_tokens, positions), offsetof(qsa_new_tokens, turn),
           offsetof(qsa_new_tokens, turn_idx), offsetof(qsa_new_tokens, eps), (int)qsa_append_tokens(0, 0, &t, 0, 0, 0),
           100 * QSA_MAX_AXES + 10 * QSA_CODE_INT4 + QSA_CODE_E2M1);
    printf("%d\n", QSA_ROWS_WORKSPACE_BYTES);
    return 0;
}
"""


def test_a_plain_c_client_includes_the_header(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    (tmp_path / "c.c").write_text(_C)
    libdir = os.path.dirname(qsa.library_path())
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", INC, str(tmp_path / "c.c"), "-o",
                    str(tmp_path / "c"), "-L", libdir, "-lqsa", "-Wl,-rpath," + libdir], check=True)
    out = subprocess.run([str(tmp_path / "c")], capture_output=True, text=True, check=True).stdout.split()
    T = qsa.QsaNewTokens
    assert [int(x) for x in out] == [
        ctypes.sizeof(qsa.QsaProjection), ctypes.sizeof(qsa.QsaRotation), ctypes.sizeof(T), T.type.offset, T.positions.offset,
        T.turn.offset, T.turn_idx.offset, T.eps.offset, INVALID,
        100 * qsa.QSA_MAX_AXES + 10 * qsa.QSA_CODE_INT4 + qsa.QSA_CODE_E2M1, qsa.QSA_ROWS_WORKSPACE_BYTES]


def test_refusals_of_the_new_tokens(lib):
    R = ctypes.byref

    def call(d=None, inp=None, tok=None, ws=F, n=256):
        return lib.qsa_append_tokens(R(d or _dims()), R(inp or _inputs()), R(tok or _tokens()), ws, n, None)

    empty = _dims(batch=0)
    assert call(d=empty) == OK
    assert call(d=_dims(group=5)) == INVALID
    assert lib.qsa_append_tokens(R(empty), None, R(_tokens()), F, 256, None) == INVALID
    assert lib.qsa_append_tokens(R(empty), R(_inputs()), None, F, 256, None) == INVALID
    assert call(n=255) == WS_SMALL and call(ws=None) == INVALID and call(ws=F + 16) == INVALID
    none = qsa.QsaProjection(None, 0, None)
    gone = {k: none for k in ("q", "k", "v", "q_idx", "idx_key")}
    assert call(d=empty, tok=_tokens(**gone)) == INVALID
    for bad in (dict(type=3), dict(type=-1), dict(axes=0), dict(axes=5), dict(eps=-1e-9), dict(eps=float("nan")), dict(positions=None),
                dict(positions=F + 2), dict(v=qsa.QsaProjection(F, 256, F)),
                dict(turn=qsa.QsaRotation(F, 132, 0)), dict(turn=qsa.QsaRotation(F, 136, 0)), dict(turn=qsa.QsaRotation(F, -8, 0)),
                dict(turn=qsa.QsaRotation(F, 12, 0)), dict(turn=qsa.QsaRotation(None, 64, 0)), dict(turn=qsa.QsaRotation(F + 2, 64, 0)),
                dict(turn=qsa.QsaRotation(F, 64, 2)), dict(turn_idx=qsa.QsaRotation(F, 72, 0)), dict(turn_idx=qsa.QsaRotation(F, 64, -1))):
        assert call(d=empty, tok=_tokens(**bad)) == INVALID, bad
    for kind, heads, width in (("q", 16, 128), ("k", 2, 128), ("v", 2, 128), ("q_idx", 8, 64), ("idx_key", 1, 64)):
        n = heads * width
        for bad in (qsa.QsaProjection(F + 8, n, None), qsa.QsaProjection(F, n - 8, None), qsa.QsaProjection(F, n + 4, None),
                    qsa.QsaProjection(F, -n, None), qsa.QsaProjection(F, 1 << 62, None)) + (
                    () if kind == "v" else (qsa.QsaProjection(F, n, F + 8),)):
            assert call(d=empty, tok=_tokens(**{kind: bad})) == INVALID, (kind, bad.rows, bad.stride)
        assert call(d=empty, tok=_tokens(**{kind: qsa.QsaProjection(F, n + 8, None)})) == OK
        assert call(d=empty, tok=_tokens(type=0, **{kind: qsa.QsaProjection(F, n + 4, None)})) == OK
        # where it goes
        dst = {"q": "q", "k": "k_cache", "v": "v_cache", "q_idx": "q_idx", "idx_key": "idx_keys"}[kind]
        for at in (None, F + 8):
            assert call(d=empty, inp=_inputs(**{dst: at})) == INVALID, kind
            others = {k: none for k in gone if k != kind}
            assert call(d=empty, inp=_inputs(**{dst: at}), tok=_tokens(**others)) == INVALID
            if kind != "v":
                assert call(d=empty, inp=_inputs(**{dst: at}), tok=_tokens(**{kind: none})) == OK
    for bad in (dict(visible=None), dict(visible=F + 2), dict(slot_map=None), dict(slot_offset=None), dict(slot_offset=F + 4),
                dict(num_slots=-1), dict(key_offset=None), dict(key_offset=F + 4)):
        assert call(d=empty, inp=_inputs(**bad)) == INVALID, bad
    # what no given projection needs may be missing, whatever it is
    q_only = _tokens(**{k: none for k in gone if k != "q"}, turn_idx=qsa.QsaRotation(None, 99, 7))
    assert call(d=empty, inp=qsa.QsaInputs(visible=F, q=F), tok=q_only) == OK
    assert call(d=_dims(batch=0, idx_dim=48), inp=qsa.QsaInputs(visible=F, q=F), tok=q_only) == OK
    idx_only = _tokens(**{k: none for k in ("q", "k", "v")}, turn=qsa.QsaRotation(None, 99, 7))
    assert call(d=_dims(batch=0, head_dim=96, q_heads=16), inp=qsa.QsaInputs(visible=F, q_idx=F, idx_keys=F, key_offset=F), tok=idx_only) == OK
    still = dict(turn=qsa.QsaRotation(None, 0, 9), turn_idx=qsa.QsaRotation(None, 0, 9), positions=None)
    assert call(d=empty, tok=_tokens(**still)) == OK
    assert call(d=_dims(head_dim=96)) == UNSUPPORTED and call(d=_dims(idx_dim=48)) == UNSUPPORTED
    # q and k alone turn: v's rotation is nobody's
    v_only = _tokens(**{k: none for k in gone if k != "v"}, turn=qsa.QsaRotation(None, 99, 7))
    assert call(d=empty, tok=v_only) == OK


def test_refusals_of_reading_back(lib):
    R = ctypes.byref

    def call(d=None, inp=None, cache=None, lo=F, hi=F, most=1, ws=F, n=256):
        return lib.qsa_read_groups(R(d or _dims()), R(inp or _inputs()), R(cache or _cache()), lo, hi, most, ws, n, None)

    only = qsa.QsaInputs(k_cache=F, v_cache=F, num_slots=1, slot_map=F, slot_offset=F)
    for fmt in (0, 1, 4, 5):
        assert call(d=_dims(batch=0), inp=only, cache=_cache(format=fmt)) == OK
        assert call(inp=only, cache=_cache(format=fmt), most=0) == OK
    assert call(d=_dims(group=5)) == INVALID and call(d=_dims(head_dim=96)) == UNSUPPORTED
    for bad in (dict(k_cache=None), dict(v_cache=None), dict(slot_map=None), dict(slot_offset=None), dict(num_slots=-1),
                dict(k_cache=F + 4), dict(slot_offset=F + 4)):
        assert call(inp=_inputs(**bad)) == INVALID, bad
    for bad in (dict(codes=None), dict(scales=None), dict(block_map=None), dict(block_offset=None), dict(num_blocks=-1),
                dict(codes=F + 8), dict(scales=F + 4), dict(format=2), dict(format=3), dict(format=6), dict(format=-1)):
        assert call(cache=_cache(**bad)) == INVALID, bad
    assert call(lo=None) == INVALID and call(hi=F + 2) == INVALID and call(most=-1) == INVALID and call(most=1025) == INVALID
    assert call(n=255) == WS_SMALL and call(ws=None) == INVALID and call(ws=F + 16) == INVALID


@pytest.mark.parametrize("fmt", [4, 5])
def test_calls_over_a_coded_cache_take_the_four_bit_formats(lib, fmt):
    R = ctypes.byref
    d = _dims(batch=0)
    c = _cache(format=fmt)
    assert lib.qsa_code_groups(R(d), R(_inputs()), R(c), F, F, 1, F, qsa.qsa_workspace_size(d), None) == OK
    n = qsa.qsa_coded_workspace_size(d, True, True)
    assert lib.qsa_attend_coded(R(d), R(_inputs()), R(c), None, None, F, F, F, F, n, None) == OK
    assert lib.qsa_decode_coded(R(d), R(_inputs()), R(c), None, None, F, F, F, None, None, F, n, None) == OK
    # the workspace does not go by the format
    assert qsa.code_bytes(fmt, 128) == 576 and qsa.code_bytes(fmt, 64) == 288 and qsa.code_bytes(qsa.QSA_CODE_INT8, 64) == 512


def test_the_binding_refuses_tensors_that_it_cannot_describe():
    import torch
    x = torch.zeros(3, 4 * 64)
    pos = torch.zeros(1, 3, dtype=torch.int32)
    f = torch.zeros(1, 32)
    ok = qsa.QsaNewTokens.of(q=x[:, :128], k=x[:, 128:].view(3, 2, 64), positions=pos[0], freq=f[0], q_norm=torch.ones(64))
    assert (ok.q.stride, ok.k.stride, ok.type, ok.axes, ok.turn.dims, ok.turn_idx.dims) == (256, 256, 0, 1, 64, 0)
    assert ok.k.rows - ok.q.rows == 512 and not ok.v.rows
    assert qsa.QsaNewTokens.of(q=x[:1, :128], positions=pos, freq=f).q.stride == 128   # of one row the heads' own width
    two = qsa.QsaNewTokens.of(q=x, positions=torch.zeros(2, 3, dtype=torch.int32), freq=torch.zeros(2, 8))
    assert two.axes == 2 and two.turn.dims == 16
    for bad in (dict(), dict(q=x.double()), dict(q=x, k=x.to(torch.bfloat16)), dict(q=x[:, ::2]), dict(q=x[0]), dict(q=x.t()),
                dict(q=x.view(3, 4, 64)[:, ::2]), dict(q=x, positions=pos.long()), dict(q=x, positions=torch.zeros(3, 1, dtype=torch.int32).t(), freq=torch.zeros(2, 8)),
                dict(q=x, positions=pos, freq=torch.zeros(2, 8)), dict(q=x, positions=pos, freq=f.double()),
                dict(q=x, positions=pos, freq=torch.zeros(1, 64)[:, ::2]), dict(q=x, k_norm=torch.ones(64)),
                dict(q=x, q_norm=torch.ones(64).half()), dict(q=x, q_norm=torch.ones(128)[::2])):
        with pytest.raises(ValueError):
            qsa.QsaNewTokens.of(**bad)


def test_the_plain_coding_is_within_half_a_step():
    """The tests' own coding against the definition: of the tile's scale t s, a value is off by at most half a
    step of its format, or by what the largest code falls short of it (t is at most 1/17 below a / (c s)); and a
    tile's scale by half a step of e4m3, 2^-4."""
    x = np.random.RandomState(0).randn(50, 4, 64).astype(np.float32)
    assert c4.e2m1_table().tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    for fmt in (c4.E2M1, c4.INT4):
        code, tile, s = c4.encode(x, fmt)
        top = c4.TOP[fmt]
        unit = np.repeat(tile * s[:, None].astype(np.float64), 4, axis=1)[:, None]
        most = np.abs(x).reshape(50, 4, 16, 4).max(axis=(1, 3)).astype(np.float64)
        assert (np.abs(tile * top * s[:, None] - most) <= 2.0 ** -4 * most * (1 + 2.0 ** -20)).all()
        step = np.maximum(np.abs(x) / unit * 2.0 ** -1, 0.5) if fmt == c4.E2M1 else np.ones_like(x)
        short = np.maximum(np.abs(x) - top * unit, 0)
        assert (np.abs(code * unit - x) <= np.maximum(step * unit / 2 * (1 + 2.0 ** -20), short * (1 + 2.0 ** -20))).all()
        allowed = set(c4.e2m1_table()) if fmt == c4.E2M1 else set(range(-7, 8))
        assert set(np.unique(code)) <= allowed


def test_rows_that_are_written_over(lib):
    """Rows that start where the call writes are refused unless they are f32 queries as they will lie."""
    R = ctypes.byref
    none = qsa.QsaProjection(None, 0, None)
    for kind, n in (("q", 2048), ("k", 256), ("v", 256), ("q_idx", 512), ("idx_key", 64)):
        for type_, stride in ((0, n), (0, n + 8), (1, n), (2, n)):
            if kind in ("q", "q_idx") and (type_, stride) == (0, n):
                continue  # allowed: it would be enqueued
            tok = dict({k: none for k in ("q", "k", "v", "q_idx", "idx_key")}, type=type_)
            tok[kind] = qsa.QsaProjection(F, stride, None)
            assert lib.qsa_append_tokens(R(_dims()), R(_inputs()), R(_tokens(**tok)), F, 256, None) == INVALID, (kind, type_, stride)
    # (more heads than a row's element count has bits for)
    assert lib.qsa_append_tokens(R(_dims(batch=0, q_heads=1 << 24, kv_heads=1 << 20)), R(_inputs()),
                                 R(_tokens(q=qsa.QsaProjection(F, 1 << 31, None), k=none, v=none)), F, 256, None) == INVALID
