"""Norms of heads whose squares are below binary32's normal range (include/qsa_rows.h: the sum of the squares may be as
small as it likes), against 64 bits with the tolerance of rows_helpers."""
import numpy as np
import pytest

import rows_helpers as rh
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


def _check(b, type_name):
    from top_group_sparse_gb300 import qsa
    t = b.on_device(type_name)
    qsa.qsa_append_tokens(t["dims"], t["inputs"], t["tokens"], t["ws"])
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    b.check(t, type_name)
    return t


@pytest.mark.parametrize("eps", [0.0, 1e-44, 2.0 ** -130, 2.0 ** -126, 1e-30, 1e-6])
@pytest.mark.parametrize("log2_size", [-48, -50, -54, -60, -63, -66, -75, -100, -126])
@pytest.mark.parametrize("d,idx_dim,type_name", [(128, 64, "f32"), (64, 32, "f32"), (128, 32, "bf16")])
def test_heads_of_every_small_size(d, idx_dim, type_name, log2_size, eps):
    need_gpu()
    _check(rh.Batch([3, 4, 9], q_heads=4, kv_heads=2, head_dim=d, idx_heads=5, idx_dim=idx_dim, seed=2, eps=eps, dims=32, idx_dims=16,
                    values=lambda r, s: np.ldexp(r.choice([-1, 1], s) * (0.5 + r.rand(*s)), log2_size).astype(np.float32)), type_name)


@pytest.mark.parametrize("pairing", [rh.HALVES, rh.NEIGHBOURS])
def test_heads_of_all_sizes_side_by_side(pairing):
    """Every head of a token another size, from subnormal numbers to 2^60: what one needs does not reach the next."""
    need_gpu()

    def values(r, s):
        x = (r.choice([-1, 1], s) * (0.5 + r.rand(*s))).reshape(s[0], -1, 32)
        return np.ldexp(x, r.randint(-140, 60, x.shape[:2] + (1,))).reshape(s).astype(np.float32)

    b = rh.Batch([5, 1, 0, 33, 2] * 50, q_heads=16, kv_heads=4, head_dim=64, idx_heads=8, idx_dim=32, seed=4, eps=0.0, values=values,
                 dims=32, pairing=pairing)
    for k in ("q", "k", "v"):  # heads of 64: both halves of a size
        x = b.fused[:, b.slice[k]].reshape(b.B, -1, 2, 32)
        x[:, :, 1] = x[:, :, 0]
    _check(b, "f32")


def test_heads_of_zeros_beside_small_ones():
    """NaN without eps, zeros with it; their neighbours as ever."""
    need_gpu()
    b = rh.Batch([3, 4], q_heads=4, kv_heads=2, head_dim=64, idx_heads=4, idx_dim=32, seed=6, eps=0.0,
                 values=lambda r, s: np.ldexp(r.randn(*s), -70).astype(np.float32))
    b.fused[0, 64:128] = 0  # q head 1
    with np.errstate(invalid="ignore"):
        want = b.expected("f32")["q"]
    t = b.on_device()
    from top_group_sparse_gb300 import qsa
    qsa.qsa_append_tokens(t["dims"], t["inputs"], t["tokens"], t["ws"])
    got = t["q"].cpu().numpy()
    assert np.isnan(got[0, 1]).all()
    keep = np.ones((2, 4), bool)
    keep[0, 1] = False
    assert (np.abs(got - want[0]) <= want[1])[keep].all()
    b.eps = 1e-40
    assert (_check(b, "f32")["q"][0, 1] == 0).all()


def test_a_head_gives_the_same_bits_beside_small_ones():
    torch = need_gpu()
    make = lambda: rh.Batch([3, 4, 9, 1], q_heads=4, kv_heads=2, head_dim=64, idx_heads=4, idx_dim=32, seed=8, eps=1e-35)
    alone, beside = make(), make()
    beside.fused[:, 64:128] *= np.float32(2.0 ** -70)     # q head 1 alone
    beside.fused[1] *= np.float32(2.0 ** -60)             # a token that shares its warps' turns with its neighbours
    a, b = _check(alone, "f32"), _check(beside, "f32")
    for name in ("q", "q_idx"):
        same = torch.ones(4, 4, dtype=torch.bool, device="cuda")
        same[1] = False
        if name == "q":
            same[:, 1] = False
        assert torch.equal(a[name][same], b[name][same])
