"""Coded caches that were made elsewhere, whose scales are of any size (include/qsa_cache.h): what blocks stand for is
a product with the scale, rounded once, and nothing on the way to it leaves binary32's range.  Against 64 bits."""
import numpy as np
import pytest

import cache4_helpers as c4
import cache_helpers as ch
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

E4M3_MAX = 0x7e  # of a tile's scale: 448


def _made_elsewhere(h, t, tiles, k_scales, v_scales, seed=1):
    """Fills every block with random codes, tile scales of the given bytes and scales of the given
    numbers; returns the values (f64) of K and V by block."""
    import torch
    r = np.random.RandomState(seed)
    d, four = h.d, h.fmt in (c4.E2M1, c4.INT4)
    shape = t["codes"].shape
    raw = r.randint(0, 256, tuple(shape)).astype(np.uint8)
    if four:
        if h.fmt == c4.INT4:  # (code + 8 is 1 .. 15)
            raw = (r.randint(1, 16, raw.shape) | r.randint(1, 16, raw.shape) << 4).astype(np.uint8)
        raw[..., 4 * d:] = r.choice(np.asarray(tiles, np.uint8), raw[..., 4 * d:].shape)
    elif h.fmt == ch.E4M3:
        raw[(raw & 0x7f) == 0x7f] = 0x7e
    s = np.stack([r.choice(np.asarray(x, np.float32), raw.shape[:2]) for x in (k_scales, v_scales)], axis=-1).astype(np.float32)
    t["codes"].copy_(torch.from_numpy(raw))
    t["scales"].copy_(torch.from_numpy(s))
    if four:
        k, v, kt, vt = c4.unpack(raw, d, h.fmt)
        k, v = (a * np.repeat(b, 4, axis=-1)[..., None, :] for a, b in ((k, kt), (v, vt)))
    else:
        k, v = ch.unpack(raw, d, h.fmt)
    return (k, v), s


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8, c4.E2M1, c4.INT4])
@pytest.mark.parametrize("kv,d", [(2, 128), (3, 64)])
def test_reading_back_with_scales_of_every_size(fmt, kv, d):
    """The largest float and powers of two on the way to it, the smallest normal and subnormal ones, zero: a value is
    the exact product rounded once, infinite only where that is beyond binary32."""
    torch = need_gpu()
    from top_group_sparse_gb300 import qsa
    four = fmt in (c4.E2M1, c4.INT4)
    h = (c4 if four else ch).History([4 * 600], q_heads=kv, kv_heads=kv, head_dim=d, fmt=fmt, seed=2)
    t = (c4 if four else ch).device(h)
    top = float(np.finfo(np.float32).max)
    sizes = [top, 2.0 ** 127, 1.7 * 2.0 ** 126, 2.0 ** 125, 1.9 * 2.0 ** 124, 2.0 ** 117, 1.0, -2.0 ** 126, 2.0 ** -126, 2.0 ** -149, 1.3e-40, 0.0]
    (k, v), s = _made_elsewhere(h, t, list(range(0, E4M3_MAX + 1)) + [0, 1, 2, 3] * 20, sizes, sizes[::-1], seed=3)
    ws = torch.zeros(qsa.QSA_ROWS_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    qsa.qsa_read_groups(t["dims"], t["inputs"], t["cache"], t["lo"], t["hi"], t["most"], ws)
    assert qsa.qsa_check_errors(ws) == (0, 0)
    slots = h.slot_map.reshape(-1, 4)
    for i, (name, x) in enumerate((("k_cache", k), ("v_cache", v))):
        with np.errstate(over="ignore"):
            want = (x * s[..., i].astype(np.float64)[..., None, None]).astype(np.float32)[h.block_map]
        got = t[name].cpu().numpy()[slots].transpose(0, 2, 1, 3)
        assert np.array_equal(got, want)
        assert np.isfinite(want).mean() > 0.5 and (np.abs(want[np.isfinite(want)]) > 2.0 ** 120).any()


@pytest.mark.parametrize("fmt", [ch.E4M3, ch.INT8, c4.E2M1, c4.INT4])
@pytest.mark.parametrize("q_heads,kv,d", [(16, 2, 128), (8, 1, 64), (16, 1, 64), (12, 1, 128)])
@pytest.mark.parametrize("whole", [True, False])
def test_attention_with_the_largest_scales(fmt, q_heads, kv, d, whole):
    """Queries of zeros over K scales up to the largest float, so that all weights are equal, and V scales just below
    2^120 with values below 2^114 (in 8 bits: scales of that size with codes up to 448): the outputs are the means.
    Tolerance: as cache_helpers.attention derives it with scores of 0, 30 * 2^-22 of the largest |v|."""
    need_gpu()
    from top_group_sparse_gb300 import qsa
    four = fmt in (c4.E2M1, c4.INT4)
    h = (c4 if four else ch).History([60, 8, 4], q_heads=q_heads, kv_heads=kv, head_dim=d, fmt=fmt, seed=4)
    h.q[:] = 0
    t = (c4 if four else ch).device(h, whole=whole)
    # 2^8 * 60 tokens * |v| < 2^128: tiles of 2^-9 .. 7 * 2^-9, codes up to 7; 8 bits without tiles: smaller scales
    v_scales = [1.9 * 2.0 ** 119, 2.0 ** 119, 2.0 ** 110] if four else [1.9 * 2.0 ** 104, 2.0 ** 104, 2.0 ** 90]
    k_scales = [float(np.finfo(np.float32).max), 2.0 ** 126, 2.0 ** 125, 1.0]
    (_, v), s = _made_elsewhere(h, t, [1, 2, 3], k_scales, v_scales, seed=5)
    V = (v * s[..., 1].astype(np.float64)[..., None, None])[h.block_map]
    ids, n = (None, None) if whole else ch.rows_to_device([np.arange(x) for x in h.visible], 512)
    qsa.qsa_attend_coded(t["dims"], t["inputs"], t["cache"], ids, n, t["out"], t["ws"])
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    got = t["out"].cpu().numpy().astype(np.float64)
    for b in range(h.B):
        x = V[h.group_offset[b]:h.group_offset[b] + h.visible[b] // 4]          # [groups, kv, 4, d]
        assert 2.0 ** 8 * np.abs(x).sum(axis=(0, 2)).max() < 2.0 ** 128
        want = np.repeat(x.mean(axis=(0, 2)), q_heads // kv, axis=0)
        assert np.abs(got[b] - want).max() <= 30 * 2.0 ** -22 * np.abs(x).max()
