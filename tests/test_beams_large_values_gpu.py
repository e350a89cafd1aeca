"""Beam selection from logits of large magnitude: rows filled with a finite mask value, and rows far from 0."""
import pytest
import torch

from test_beams_gpu import INF, _candidates, _check, _logits

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FAR = [s * m for m in (3e3, 1e5, 1e6, 1e7, 1e8, 1e9, 1e12, 1e30) for s in (1.0, -1.0)]


def _rows(V, dtype, seed=0):
    z, s = _logits(8, V, dtype, V + seed)
    return z, s


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("V", [1000, 20001])
def test_a_row_filled_with_one_value(lmh, V, far, dtype):
    """A row of equal logits beside healthy ones: each of its tokens has the log-probability -log V, and the other
    beams keep their continuations."""
    if dtype == F16 and abs(far) > 6e4:
        far = 6e4 if far > 0 else -6e4
    z, s = _rows(V, dtype)
    z[1] = far
    z[6] = far
    s[6] = 2.0  # this one leads its group
    for k in (4, 8):
        _check(lmh.beam_select(z, s, 4, k=k), _candidates(z, s, 4), 4, k)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("far", FAR)
def test_a_healthy_row_moved(lmh, far, dtype):
    """Logits that lie around a large value (as far as the type tells them apart)."""
    if dtype == F16 and abs(far) > 6e4:
        far = 6e4 if far > 0 else -6e4
    z, s = _rows(6001, F32)
    z[2] = z[2] * max(1.0, abs(far) * torch.finfo(dtype).eps) + far
    z[5] += far
    z = z.to(dtype)
    s[2] = s[5] = 0.5
    _check(lmh.beam_select(z, s, 4, k=8), _candidates(z, s, 4), 4, 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fill", [-1e4, -1e9, -1e30])
@pytest.mark.parametrize("V", [4099, 50000])
def test_tokens_masked_by_a_finite_value(lmh, V, fill, dtype):
    """In place of a mask: all tokens but a few, in runs and alone, of every row, and of one row all."""
    z, s = _rows(V, dtype, 1)
    keep = torch.zeros(V, dtype=torch.bool, device="cuda")
    keep[[0, 5, 63, 64, 900, V - 1]] = True
    keep[1000:1130] = True
    z[:, ~keep] = fill
    z[3] = fill
    _check(lmh.beam_select(z, s, 4, k=8), _candidates(z, s, 4), 4, 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_values_beside_infinities_and_nan(lmh, dtype):
    z, s = _rows(9000, dtype, 2)
    z[0], z[1], z[2] = -1e9, 1e9, 1e12
    z[0, ::5] = float("nan")
    z[1, 3::7] = -INF
    z[2, 40:90] = float("nan")
    z[4] = -1e9
    z[4, 100:200] = INF
    _check(lmh.beam_select(z, s, 4, k=8), _candidates(z, s, 4), 4, 8)


@pytest.mark.parametrize("far", [-1e4, -1e9, -1e30])
@pytest.mark.parametrize("dtype,V", [(F32, 5003), (BF16, 30000), (F32, 151936), (BF16, 248320)])
def test_a_search_that_begins(lmh, V, dtype, far):
    """The first step of a search: rows alike, all beams but a group's first far below."""
    z = _logits(2, V, dtype, 5)[0].repeat_interleave(4, 0).contiguous()
    s = torch.full((8,), far, device="cuda")
    s[0] = s[4] = 0.0
    _check(lmh.beam_select(z, s, 4, k=8), _candidates(z, s, 4), 4, 8)
    keep = lmh.beam_select(z, s, 4, keep_slots=True)
    _check(keep, _candidates(z, s, 4), 4, 4, keep=True)


def _choice_ms(lmh, z, s):
    """The choice kernel's shortest time of ten calls."""
    from top_reduction_gb300 import lmh as L
    best = INF
    L.trace_enable(True)
    try:
        for _ in range(10):
            L.trace_reset()
            lmh.beam_select(z, s, 4, k=8)
            best = min(best, L.trace_read("beam_choose")[1])
    finally:
        L.trace_enable(False)
        L.trace_reset()
    return best


@pytest.mark.parametrize("dtype,V", [(F32, 151936), (BF16, 248320)])
def test_a_search_that_begins_takes_a_usual_steps_time(lmh, V, dtype):
    """Beams far below do not widen what the choice looks through: nine blocks of ten are sorted out as in any step.
    (Looked through one by one a group's logits take hundreds of times as long.)"""
    z, s = _logits(4, V, dtype, 6)
    usual = _choice_ms(lmh, z, s)
    s[1:] = -1e9
    assert _choice_ms(lmh, z, s) <= 3 * usual


def test_scores_above_0(lmh):
    """A leader far above the others, alone or with fewer tokens than are asked for."""
    for k in (2, 8):
        z, s = _logits(8, 3001, F32, 7)
        s[1], s[6] = 5e4, 300.0
        z[1, 3:] = -INF
        z[6, 1:] = -INF
        _check(lmh.beam_select(z, s, 4, k=k), _candidates(z, s, 4), 4, k)
