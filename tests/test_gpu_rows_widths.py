"""qsa_append_tokens for every pair of head widths, type and kind of rotation (tests/rows_helpers.py)."""
import pytest

import rows_helpers as rh
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type_name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,idx_dim", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("pairing", [rh.HALVES, rh.NEIGHBOURS])
def test_every_pair_of_widths(d, idx_dim, type_name, pairing):
    need_gpu()
    from top_group_sparse_gb300 import qsa
    for dims, idx_dims, norms in ((d, idx_dim, True), (24, 8, False), (d - 8, 24, True), (0, idx_dim, True)):
        b = rh.Batch([5, 1, 0, 33, 2, 7, 8], q_heads=7, kv_heads=1, head_dim=d, idx_heads=3, idx_dim=idx_dim, seed=9, axes=3, pairing=pairing,
                     idx_pairing=1 - pairing, dims=dims, idx_dims=idx_dims, norms=norms, pad=16)
        t = b.on_device(type_name)
        qsa.qsa_append_tokens(t["dims"], t["inputs"], t["tokens"], t["ws"])
        assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
        b.check(t, type_name)
