"""What add_adapters keeps of the adapters' part where 16-bit outputs are small beside it."""
import pytest
import torch

from test_adapters_gpu import BF16, F16, F32, _case, _formula, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,H,N,R,L", [
    (1, 256, 512, 16, 2), (6, 128, 333, 8, 2), (33, 512, 1000, 32, 4), (64, 128, 260, 64, 3), (130, 128, 516, 128, 3),
    (300, 128, 512, 16, 2), (300, 64, 1001, 32, 3), (513, 256, 1028, 64, 4), (700, 64, 264, 128, 3)])
def test_parts_that_cancel(lmh, rows, H, N, R, L, dtype):
    """y takes nearly all of the adapter's part away: what is left is off by the fp32 sums' roundings, by d's second
    part's (2^-16 of d for bf16, 2^-22 for f16) and by its own last one, not by a rounding of d to 16 bits."""
    c = _case(rows, H, N, R, L, dtype, F32, seed=rows + R, none=False)
    c["y"] = torch.zeros(rows, N, dtype=F32, device="cuda")
    part, _ = _formula(c)
    c["y"] = (-part).to(dtype)
    got = _run(lmh, c)
    assert got.dtype == dtype
    want, off = _formula(dict(c, y=c["y"].float()))
    off = off + (want.abs() + off) * (2.0 ** -24 + torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == F16 else 0)
    bad = ~((got.double() - want).abs() <= off)
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()), float(off.max()))


@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("N", [40, 44, 33])
@pytest.mark.parametrize("rows", [5, 20, 300])
def test_rows_that_nothing_is_added_to(lmh, rows, N, dtype, y_dtype):
    """A row without an adapter, or with one of rank 0, is y to the sign of its zeros."""
    c = _case(rows, 64, N, 16, 3, dtype, y_dtype, seed=N)
    c["ranks"] = torch.tensor([0, 16, 5], dtype=torch.int32, device="cuda")
    c["idx"][0], c["idx"][1], c["idx"][2] = -1, 0, 1
    c["y"][:, ::3] = -0.0
    c["y"][:, 1::3] = 0.0
    got = _run(lmh, c)
    same = c["idx"] <= 0
    bits = torch.int32 if y_dtype == F32 else torch.int16
    assert torch.equal(got[same].view(bits), c["y"][same].view(bits))
