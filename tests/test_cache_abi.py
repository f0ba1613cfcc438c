"""include/qsa_cache.h: every declared symbol is exported, sizes have their
closed forms, a plain C client compiles against the header, and every refusal
that the host can make is made before anything is enqueued (no GPU here: a call
that enqueued something would fail)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import cache_helpers as ch
from top_group_sparse_gb300 import build as qbuild
from top_group_sparse_gb300 import qsa

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
INC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(qsa.__file__))), "include")
CALLS = ["qsa_attend_coded", "qsa_code_groups", "qsa_coded_workspace_size", "qsa_decode_coded", "qsa_evict_compact",
         "qsa_evict_select"]
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
    base = dict(codes=F, scales=F, num_blocks=100, block_map=F, block_offset=F, format=0)
    base.update(kw)
    return qsa.QsaCodedCache(**base)


def _hist(at=F, **kw):
    base = {n: at for n, _ in qsa.QsaHistory._fields_}
    base.update(kw)
    return qsa.QsaHistory(**base)


def test_every_declared_symbol_is_exported(lib):
    assert qsa.exported_symbols(os.path.join(INC, "qsa_cache.h")) == CALLS
    for n in CALLS:
        assert hasattr(lib, n) and n in qsa.__all__


def test_workspace_closed_forms(lib):
    def up(x):
        return (x + 255) // 256 * 256

    d = _dims()
    base = qsa.qsa_workspace_size(d)
    assert qsa.qsa_coded_workspace_size(d, False, False) == base
    heads = 2 * 16
    # 1,024 groups: 16 runs of 64, and the tail's
    part = 2 * up(heads * 17 * 4) + up(heads * 17 * 128 * 4)
    assert qsa.qsa_coded_workspace_size(d, True, False) == base + part
    mass = up(heads * 1024 * 4) + up(heads * 256 * 4) + up(heads * 8) + 2 * up(2 * 4)
    assert qsa.qsa_coded_workspace_size(d, True, True) == base + part + mass
    rows = up(heads * 512 * 4) + up(heads * 128 * 4) + up(heads * 8) + 2 * up(2 * 4)
    assert qsa.qsa_coded_workspace_size(d, False, True) == base + rows
    # the longest history: at most 512 runs and the tail's, whatever its length
    d = _dims(batch=1, max_visible=1 << 26)
    assert qsa.qsa_coded_workspace_size(d, True, False) - qsa.qsa_workspace_size(d) == \
        2 * up(16 * 513 * 4) + up(16 * 513 * 128 * 4)
    assert qsa.qsa_coded_workspace_size(_dims(group=3), True, True) == 0


def test_a_longer_history_needs_no_smaller_workspace(lib):
    """A workspace made for max_visible serves every shorter row, whose cut into
    runs may be finer."""
    last = 0
    for t in sorted({g * 4 + o for g in (1, 31, 32, 1023, 1024, 1025, 2048, 4096, 4097, 8192, 65535, 65536, 65537, 100000)
                     for o in (0, 3)}):
        n = qsa.qsa_coded_workspace_size(_dims(max_visible=t), True, False) - qsa.qsa_workspace_size(_dims(max_visible=t))
        assert n >= last, t
        last = n


def test_refusals_of_the_coding(lib):
    d, R = _dims(), ctypes.byref
    need = qsa.qsa_workspace_size(d)

    def call(d=d, inp=None, cache=None, lo=F, hi=F, most=1, ws=F, n=need):
        return lib.qsa_code_groups(R(d), R(inp or _inputs()), R(cache or _cache()), lo, hi, most, ws, n, None)

    assert call(d=_dims(group=5)) == INVALID
    assert call(d=_dims(head_dim=96)) == UNSUPPORTED
    for bad in (dict(k_cache=None), dict(v_cache=None), dict(slot_map=None), dict(slot_offset=None), dict(num_slots=-1),
                dict(k_cache=F + 4), dict(slot_offset=F + 4)):
        assert call(inp=_inputs(**bad)) == INVALID, bad
    for bad in (dict(codes=None), dict(scales=None), dict(block_map=None), dict(block_offset=None), dict(num_blocks=-1),
                dict(codes=F + 8), dict(scales=F + 4), dict(format=2), dict(format=-1)):
        assert call(cache=_cache(**bad)) == INVALID, bad
    assert call(lo=None) == INVALID and call(hi=F + 2) == INVALID
    assert call(most=-1) == INVALID and call(most=1025) == INVALID
    assert call(n=need - 1) == WS_SMALL and call(ws=None) == INVALID and call(ws=F + 16) == INVALID
    # the raw cache alone is read: the other members may be NULL
    only = qsa.QsaInputs(k_cache=F, v_cache=F, num_slots=1, slot_map=F, slot_offset=F)
    assert lib.qsa_code_groups(R(_dims(batch=0)), R(only), R(_cache()), F, F, 1, F, need, None) == OK


def test_refusals_of_the_attention(lib):
    d, R = _dims(), ctypes.byref
    need = qsa.qsa_coded_workspace_size(d, True, True)

    def call(d=d, inp=None, cache=None, ids=F, n_ids=F, out=F, w=None, wo=None, ws=F, n=need):
        return lib.qsa_attend_coded(R(d), R(inp or _inputs()), R(cache or _cache()), ids, n_ids, out, w, wo, ws, n, None)

    assert call(d=_dims(budget_groups=513)) == INVALID
    assert call(d=_dims(head_dim=96)) == UNSUPPORTED and call(d=_dims(q_heads=64)) == UNSUPPORTED
    for bad in (dict(q=None), dict(q=F + 4), dict(visible=None), dict(k_cache=None), dict(slot_map=None)):
        assert call(inp=_inputs(**bad)) == INVALID, bad
    assert call(cache=_cache(format=7)) == INVALID and call(cache=_cache(codes=None)) == INVALID
    assert call(ids=None) == INVALID and call(n_ids=None) == INVALID and call(ids=F + 2) == INVALID
    assert call(out=None) == INVALID and call(out=F + 4) == INVALID
    assert call(w=F) == INVALID and call(wo=F) == INVALID and call(w=F + 2, wo=F) == INVALID
    for ids, w in ((F, None), (F, F), (None, None), (None, F)):
        least = qsa.qsa_coded_workspace_size(d, ids is None, w is not None)
        assert call(ids=ids, n_ids=ids, w=w, wo=w, n=least - 1) == WS_SMALL
        empty = _dims(batch=0)
        assert call(d=empty, ids=ids, n_ids=ids, w=w, wo=w) == OK


def test_refusals_of_the_whole_path(lib):
    d, R = _dims(), ctypes.byref
    need = qsa.qsa_coded_workspace_size(d, False, True)

    def call(d=d, inp=None, pooled=None, po=None, ids=F, n_ids=F, out=F, w=None, wo=None, n=need):
        return lib.qsa_decode_coded(R(d), R(inp or _inputs()), R(_cache()), pooled, po, ids, n_ids, out, w, wo, F, n, None)

    assert call(d=_dims(idx_dim=48)) == UNSUPPORTED and call(d=_dims(head_dim=96)) == UNSUPPORTED
    assert call(inp=_inputs(q_idx=None)) == INVALID and call(inp=_inputs(idx_keys=None)) == INVALID
    assert call(inp=_inputs(key_offset=None)) == INVALID
    assert call(pooled=F) == INVALID and call(po=F) == INVALID and call(pooled=F + 4, po=F) == INVALID
    assert call(ids=None) == INVALID and call(n_ids=None) == INVALID and call(out=F + 8) == INVALID and call(w=F) == INVALID
    assert call(n=qsa.qsa_coded_workspace_size(d, False, False) - 1) == WS_SMALL
    assert call(w=F, wo=F, n=need - 1) == WS_SMALL
    assert call(d=_dims(batch=0)) == OK
    assert call(d=_dims(batch=0), inp=_inputs(idx_keys=None, key_offset=None), pooled=F, po=F) == OK


def test_refusals_of_the_eviction(lib):
    d, R = _dims(), ctypes.byref
    need = qsa.qsa_workspace_size(d)

    def sel(d=d, vis=F, w=F, wo=F, keep=8, sink=1, recent=2, kept=F, n_kept=F, ev=None, n=need):
        return lib.qsa_evict_select(R(d), vis, w, wo, keep, sink, recent, kept, n_kept, ev, F, n, None)

    for bad in (dict(vis=None), dict(w=None), dict(wo=None), dict(kept=None), dict(n_kept=None), dict(keep=0),
                dict(keep=(1 << 24) + 1), dict(sink=-1), dict(recent=-1), dict(sink=9), dict(sink=7, recent=2),
                dict(recent=2 ** 31 - 1), dict(w=F + 2), dict(wo=F + 4), dict(ev=F + 1), dict(d=_dims(group=2))):
        assert sel(**bad) == INVALID, bad
    assert sel(n=need - 1) == WS_SMALL and sel(d=_dims(batch=0)) == OK

    def mov(d=d, keep=8, kept=F, n_kept=F, src=None, dst=None, n=need):
        return lib.qsa_evict_compact(R(d), keep, kept, n_kept, R(src or _hist()), R(dst or _hist(2 * F)), F, n, None)

    assert mov(d=_dims(idx_dim=48)) == UNSUPPORTED
    assert mov(keep=0) == INVALID and mov(kept=None) == INVALID and mov(n_kept=None) == INVALID
    assert mov(dst=_hist(F)) == INVALID  # in place
    for name in ("idx_keys", "pooled", "slot_map", "block_map", "weights"):
        assert mov(dst=_hist(2 * F, **{name: None})) == INVALID, name  # one side only
        assert mov(src=_hist(F, **{name: None})) == INVALID, name
        assert mov(dst=_hist(2 * F, **{name: F})) == INVALID, name     # the same array
        assert mov(dst=_hist(2 * F, **{name: 2 * F + 2})) == INVALID, name
    for name in ("key_offset", "pool_offset", "slot_offset", "block_offset", "weight_offset"):
        assert mov(dst=_hist(2 * F, **{name: None})) == INVALID, name
    assert mov(src=_hist(F, visible=None)) == INVALID and mov(dst=_hist(2 * F, visible=None)) == INVALID
    assert mov(n=need - 1) == WS_SMALL and mov(d=_dims(batch=0)) == OK
    # what neither history has is not moved
    none = {n: None for n in ("pooled", "pool_offset", "weights", "weight_offset")}
    assert mov(d=_dims(batch=0), src=_hist(F, **none), dst=_hist(2 * F, **none)) == OK


_C = r"""
#include <stdio.h>
#include "qsa_cache.h"

int main(void)
{
    qsa_dims d = {2, 8, 64, 16, 2, 128, 4, 512, 4096, 0.088388347648f};
    qsa_coded_cache c = {0};
    qsa_history h = {0};
    c.format = QSA_CODE_INT8;
    printf("%zu %zu %d\n", qsa_coded_workspace_size(&d, 1, 1), sizeof c + 0 * sizeof h, (int)qsa_evict_compact(&d, 1, 0, 0, &h, &h, 0, 0, 0));
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
    assert int(out[0]) == qsa.qsa_coded_workspace_size(_dims(), True, True)
    assert int(out[1]) == ctypes.sizeof(qsa.QsaCodedCache) and int(out[2]) == INVALID


def test_the_plain_coding_is_within_half_a_step(lib):
    """The tests' own coding, against the definition: a value is off by at most
    half a step of its format (e4m3: 2^-4 of the value or half the smallest
    step, int8: half a code), and the table has the format's extremes."""
    t = ch.e4m3_table()
    assert np.nanmax(t) == 448 and np.isnan(t[[0x7f, 0xff]]).all() and t[1] == 2.0 ** -9
    x = np.random.RandomState(0).randn(50, 4, 64).astype(np.float32)
    for fmt in (0, 1):
        c, s = ch.encode(x, fmt)
        err = np.abs(c * s[:, None, None].astype(np.float64) - x)
        step = np.maximum(np.abs(x) * 2.0 ** -4, s[:, None, None] * 2.0 ** -10) if fmt == 0 else s[:, None, None] * 0.5
        assert (err <= step * (1 + 2.0 ** -20)).all()
        assert set(np.unique(c)) <= set(t[~np.isnan(t)] if fmt == 0 else range(-127, 128))


def test_the_plain_eviction_keeps_what_the_definition_says(lib):
    w = np.array([5, 0, 0, 3, np.nan, 0, 9, -np.inf, 1, 2], np.float32)
    assert ch.evict([40], w, [0], 6, 1, 2)[0].tolist() == [0, 1, 3, 6, 8, 9]
    assert ch.evict([43], w, [0], 10, 0, 0)[0].tolist() == list(range(10))
    assert ch.evict([40], w, [0], 9, 0, 0)[0].tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]  # the NaN goes first
