"""lmh_project_q4 with and without zero points, on both sides of 16 hidden rows: gathered rows, strides,
extreme and non-finite hidden values, long hidden rows.

More than 16 rows without zero points run on another kernel than the rest.  Bounds as in test_q4_gpu.py:
(H + 8) * 2^-23 of the sum of the terms' magnitudes.
"""
import math

import numpy as np
import pytest
import torch

from test_q4_gpu import DT, check_project, random_table

pytestmark = pytest.mark.gpu

ROWS = [11, 24]
BOTH = pytest.mark.parametrize("zeros", [False, True])


@BOTH
@pytest.mark.parametrize("n", ROWS + [33, 50])
@pytest.mark.parametrize("scale", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_strides_and_row_index(lmh, n, zeros, scale, out):
    """Hidden rows at odd and even strides, table rows and output rows with spare columns; indices out of range in
    both halves of a pass read zeros and set the status bit; nothing is written beside the output's columns."""
    rng = np.random.default_rng(n)
    V, H, T = 777, 320, 50
    table, w = random_table(lmh, V, H, 32, zeros, scale=scale, seed=3, pad=3)
    bad = [1, 3, n - 2]
    for pad, first in [(0, 0), (3, 1), (8, 8), (1, 0)]:
        full = torch.from_numpy(rng.standard_normal((T, first + H + pad)).astype(np.float32)).to(torch.bfloat16).cuda()
        hidden = full[:, first:first + H]
        idx = rng.integers(0, T, n).astype(np.int32)
        idx[bad] = [-1, T, 2 ** 31 - 1]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        buf = torch.full((n, V + 5), 7.0, device="cuda", dtype=DT[out])
        lmh.project_q4(hidden, table, row_idx=torch.from_numpy(idx).cuda(), out=buf[:, 2:2 + V], dev_status=status)
        x = hidden.double().cpu().numpy()[np.clip(idx, 0, T - 1)]
        x[bad] = 0
        check_project(buf[:, 2:2 + V], x, w, H, 1.0, out)
        assert (buf[bad, 2:2 + V] == 0).all()
        assert (buf[:, :2] == 7).all() and (buf[:, 2 + V:] == 7).all()
        assert int(status.item()) == 0x8
        good = np.setdiff1d(np.arange(n), bad)
        status.zero_()
        lmh.project_q4(hidden, table, row_idx=torch.from_numpy(idx[good]).cuda(), dev_status=status)
        assert int(status.item()) == 0


@BOTH
@pytest.mark.parametrize("rows", [16, 24, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_hidden_ranges(lmh, dtype, rows, zeros):
    """Rows of very large, very small, subnormal and widely spread values, and zeros, in both halves of a pass."""
    rng = np.random.default_rng(31)
    V, H = 400, 640
    table, w = random_table(lmh, V, H, 64, zeros, scale="f32", seed=9)
    big, small = (1e30, 1e-36) if dtype == "bf16" else (3e4, 1e-7)
    x = rng.standard_normal((rows, H))
    lim = 6e4 if dtype == "f16" else 3e38
    for base in {0, rows - 8}:
        for i, f in enumerate([big, small, 1e-40 if dtype == "bf16" else 6e-8, 0.0]):
            x[base + i] = np.clip(x[base + i] * f, -lim, lim)
        x[base + 4] *= 10.0 ** rng.uniform(-20 if dtype == "bf16" else -4, 4, H)
        x[base + 5, ::2] = 0
        x[base + 6] = 0
        x[base + 6, 17] = 1.5
        x[base + 7] = np.where(np.arange(H) == 5, -lim, 0)
    xt = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    check_project(lmh.project_q4(xt, table), xt.double().cpu().numpy(), w, H, 1.0, "f32")


@BOTH
@pytest.mark.parametrize("rows", ROWS + [32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_infinities_and_nan_stay_in_their_row(lmh, rows, group, zeros):
    """A row with one infinity has that infinity times the entry at its place (NaN where the entry is 0), a row
    with a NaN is NaN, and the other rows are what they are without them."""
    V, H = 300, 512
    table, w = random_table(lmh, V, H, group, zeros, seed=5)
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(rows, H, generator=gen, device="cuda").to(torch.bfloat16)
    clean = lmh.project_q4(x, table)
    nan, plus, minus = [2, rows - 3], [5, rows - 1], [0, rows - 4]
    at = 3
    for r in nan:
        x[r, 100] = math.nan
    for r in plus:
        x[r, at] = math.inf
    for r in minus:
        x[r, at] = -math.inf
    out = lmh.project_q4(x, table).cpu().numpy()
    assert np.isnan(out[nan]).all()
    with np.errstate(invalid="ignore"):
        want = np.where(w[:, at] == 0, np.nan, np.sign(w[:, at]) * np.inf).astype(np.float32)
    for r in plus:
        np.testing.assert_array_equal(out[r], want)
    for r in minus:
        np.testing.assert_array_equal(out[r], -want)
    good = [i for i in range(rows) if i not in nan + plus + minus]
    assert np.array_equal(out[good], clean.cpu().numpy()[good])
    fresh = torch.randn(rows, H, generator=gen.manual_seed(6), device="cuda").to(torch.bfloat16)
    check_project(clean, fresh.double().cpu().numpy(), w, H, 1.0, "f32")


@BOTH
@pytest.mark.parametrize("rows,H,group", [(1, 16384, 128), (8, 9984, 64), (9, 8192, 64), (32, 8192, 32), (20, 13824, 128),
                                          (4, 14336, 32), (24, 2816, 32), (24, 2944, 128), (17, 5120, 64),
                                          (12, 5376, 128)])
def test_long_rows(lmh, rows, H, group, zeros):
    """Hidden rows about as long as shared memory holds, and longer ones that it takes in pieces."""
    rng = np.random.default_rng(H)
    table, w = random_table(lmh, 700, H, group, zeros, seed=H)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = lmh.project_q4(x, table)
    check_project(out, x.double().cpu().numpy(), w, H, 1.0, "f32")
    assert torch.equal(lmh.project_q4(x, table), out)
