"""Beam selection with ended beams: their logits are not read."""
import pytest
import torch

from test_beams_gpu import INF, _candidates, _check, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["first", "last", "all but one", "all", "none"])
@pytest.mark.parametrize("groups,V", [(1, 100), (3, 9001), (20, 60001)])
def test_runs_of_ended_beams(lmh, groups, V, which, dtype):
    """A stream's first chunks, its last ones, or all of them belong to ended beams."""
    rows = groups * 4
    z, s = _logits(rows, V, dtype, groups)
    r = torch.arange(rows, device="cuda")
    done = {"first": r < (rows + 1) // 2, "last": r >= rows // 2, "all but one": r != 2, "all": r >= 0, "none": r < 0}[which]
    z[done] = INF
    o = lmh.beam_select(z, s, 4, finished=done, pad_id=3)
    _check(o, _candidates(z, s, 4, finished=done, pad=3), 4, 4, pad=3, finished=done)


def _stream_ms(lmh, z, s, done):
    """The stream kernel's shortest time of thirty calls."""
    from top_reduction_gb300 import lmh as L
    best = INF
    L.trace_enable(True)
    try:
        for _ in range(30):
            L.trace_reset()
            lmh.beam_select(z, s, 4, finished=done)
            best = min(best, L.trace_read("beam_stream")[1])
    finally:
        L.trace_enable(False)
        L.trace_reset()
    return best


def test_ended_beams_cost_no_reads(lmh):
    """50 MB of logits that one call reads and another, whose beams have all ended, does not: 0.51 to 0.60 of the time,
    all of it the launch's; 0.83 where every CTA reads its first three chunks whatever the flags."""
    z, s = _logits(96, 128256, torch.float32, 1)
    none = torch.zeros(96, dtype=torch.uint8, device="cuda")
    assert _stream_ms(lmh, z, s, none + 1) <= 0.72 * _stream_ms(lmh, z, s, none)
