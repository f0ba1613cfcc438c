"""The angles of qsa_append_tokens read out of what it writes: f32 rows without norms whose pairs are (1, 0) come back
as (cos, sin).  Against integers and 64 bits (include/qsa_rows.h states the bounds)."""
import numpy as np
import pytest

import rows_helpers as rh
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

TWO_PI_DIGITS = 6283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136  # * 10^-99


def exact_turns(positions, freq):
    """The fraction of a turn, -1/2 .. 1/2, of one angle: positions [axes] and freq [axes] (binary32), in units of
    2^-100."""
    n, low = 0, -200
    for p, f in zip(positions, freq):
        m, e = np.frexp(np.float64(f))
        n += int(p) * (int(m * 2 ** 24) << (int(e) - 24 - low))
    one = 1 << 100
    t = (n * 10 ** 99 * one // (TWO_PI_DIGITS << -low)) % one
    return t - one if 2 * t > one else t


def _read_out(positions, freq, pairing=rh.HALVES):
    """(cos, sin) [B, pairs] f32 of positions [axes, B] and freq [axes, 32], as the call makes them."""
    import torch
    from top_group_sparse_gb300 import qsa
    B = positions.shape[1]
    x = np.zeros((B, 64), np.float32)
    one, two = (slice(0, 32), slice(32, 64)) if pairing == rh.HALVES else (slice(0, 64, 2), slice(1, 64, 2))
    x[:, one] = 1
    t = {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in
         dict(x=x, positions=positions, freq=freq, visible=np.ones(B, np.int32)).items()}
    out = torch.full((B, 1, 64), -9.0, device="cuda")
    ws = torch.zeros(qsa.QSA_ROWS_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    tok = qsa.QsaNewTokens.of(q=t["x"], positions=t["positions"], freq=t["freq"], pairing=pairing)
    qsa.qsa_append_tokens(qsa.make_dims(B, 4, 32, 1, 1, 64, max_visible=1),
                          qsa.QsaInputs(visible=t["visible"].data_ptr(), q=out.data_ptr()), tok, ws)
    assert qsa.qsa_check_errors(ws) == (0, 0)
    y = out.cpu().numpy()[:, 0]
    return y[:, one], y[:, two]


def _positions_of_small_angles(freq, tokens, seed):
    """Positions [axes, tokens] all over 32 bits for which the angle of pair b % 32 is less than 2^-15 of a turn from a
    whole number of turns (found modulo 2^64, with frequencies to 2^-64)."""
    r = np.random.RandomState(seed)
    axes = len(freq)
    unit = [[(int(np.frexp(np.float64(f))[0] * 2 ** 24) * 10 ** 99 * 2 ** 64 * 2 ** 200 >> (200 + 24 - int(np.frexp(np.float64(f))[1]))) // TWO_PI_DIGITS
             for f in row] for row in freq]
    out = np.zeros((axes, tokens), np.int32)
    for b in range(tokens):
        j = b % 32
        p = r.randint(-2 ** 31, 2 ** 31, axes, dtype=np.int64)
        last = r.randint(-2 ** 31, 2 ** 31, 1 << 18, dtype=np.int64)
        base = sum(int(p[a]) * unit[a][j] for a in range(axes - 1)) % 2 ** 64
        turn = last.astype(np.uint64) * np.uint64(unit[-1][j] % 2 ** 64) + np.uint64(base)
        p[-1] = last[np.argmin(np.abs(turn.view(np.int64)))]
        out[:, b] = p
    return out


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_the_fraction_of_a_turn_whatever_the_position(axes):
    """Angles next to whole turns: the sine is the angle itself there (to a sixth of its cube), so it shows to what
    fraction of a turn the angle was kept, (axes + 3) * 2^-34.  What the sine adds: 2^-24 of it for the angle's
    conversion, its factor, the factor's own rounding and the series' last sum, 4 * 2^-24 of less than 2^-15 of a turn."""
    need_gpu()
    r = np.random.RandomState(axes)
    freq = (r.choice([-1, 1], (axes, 32)) * np.exp(r.uniform(np.log(1e-3), np.log(60000.0), (axes, 32)))).astype(np.float32)
    positions = _positions_of_small_angles(freq, 320, 7 + axes)
    _, sine = _read_out(positions, freq)
    worst = 0.0
    for b in range(320):
        j = b % 32
        turn = exact_turns(positions[:, b], freq[:, j]) / 2.0 ** 100
        assert abs(turn) < 2.0 ** -15
        angle = turn * rh.TWO_PI
        err = abs(float(sine[b, j]) - np.sin(angle)) / rh.TWO_PI
        worst = max(worst, (err - 4 * 2.0 ** -24 * abs(turn)) * 2.0 ** 34)
    assert worst <= axes + 3, worst


@pytest.mark.parametrize("pairing", [rh.HALVES, rh.NEIGHBOURS])
@pytest.mark.parametrize("far", [1000, 2 ** 31])
def test_sines_and_cosines_to_two_to_the_minus_22(far, pairing):
    """64,000 angles all over the turn."""
    need_gpu()
    r = np.random.RandomState(3)
    freq = np.exp(r.uniform(np.log(0.01), np.log(100.0), (1, 32))).astype(np.float32)
    positions = r.randint(-far, far, (1, 2000), dtype=np.int64).astype(np.int32)
    c, s = _read_out(positions, freq, pairing)
    want = rh.angles(positions, freq)
    assert np.abs(c - np.cos(want)).max() <= 2.0 ** -22
    assert np.abs(s - np.sin(want)).max() <= 2.0 ** -22
    # the whole of a turn's quarters, their ends among them
    x = np.abs(want / rh.TWO_PI * 4 - np.rint(want / rh.TWO_PI * 4))
    assert x.max() > 0.4999 and x.min() < 1e-4


@pytest.mark.parametrize("type_name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pairing", [rh.HALVES, rh.NEIGHBOURS])
@pytest.mark.parametrize("dims,idx_dims", [(128, 64), (72, 40), (16, 8), (24, 56)])
def test_turned_rows_without_norms(dims, idx_dims, pairing, type_name):
    """A turned element is two products with a sine and a cosine that are off by 2^-22, and their sum: 6 * 2^-24 of
    |y_i| + |y_k| (rows_helpers derives it), a quarter of what that allows where a norm may come before it."""
    need_gpu()
    from top_group_sparse_gb300 import qsa
    b = rh.Batch([7, 3, 1, 0, 20], q_heads=6, kv_heads=2, head_dim=128, idx_heads=5, idx_dim=64, seed=5, norms=False, dims=dims,
                 idx_dims=idx_dims, pairing=pairing, axes=3, far=1 << 30)
    t = b.on_device(type_name)
    qsa.qsa_append_tokens(t["dims"], t["inputs"], t["tokens"], t["ws"])
    assert qsa.qsa_check_errors(t["ws"]) == (0, 0)
    want = b.expected(type_name)
    has, row, slot = b.places()
    for kind, name, at in (("q", "q", np.flatnonzero(has)), ("k", "k_cache", slot), ("q_idx", "q_idx", np.flatnonzero(has)),
                           ("idx_key", "idx_keys", row)):
        y, tol = want[kind]
        got = t[name].cpu().numpy().reshape(t[name].shape[0], -1, b.width[kind])[at].astype(np.float64)
        assert (np.abs(got - y[has]) <= tol[has] / 4).all(), kind
