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
