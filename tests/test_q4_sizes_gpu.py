"""lmh_project_q4 at the ends of its sizes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,H,zeros", [(8 * 65535 + 9, 8192, False),   # passes of 8 hidden rows
                                          (16 * 65535 + 21, 2816, True),  # of 16
                                          (32 * 65535 + 40, 64, True), (32 * 65535 + 40, 64, False)])  # of 32
@pytest.mark.parametrize("by_index", [True, False])
def test_more_passes_than_a_grid_holds(lmh, rows, H, zeros, by_index):
    """A row's logits are the same, bit for bit, wherever it stands among however many others."""
    if not by_index and H > 64:
        pytest.skip("the same launches as by index, with gigabytes of hidden rows")
    V, T = 24, 50
    gen = torch.Generator("cuda").manual_seed(H)
    table = lmh.quantize_q4(torch.randn(V, H, generator=gen, device="cuda").to(torch.bfloat16), 32, zeros=zeros)
    x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
    few = lmh.project_q4(x, table)
    idx = torch.randint(0, T, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    idx[-1] = T  # out of range: zeros, and the status bit
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if by_index:
        out = lmh.project_q4(x, table, row_idx=idx, dev_status=status)
        assert int(status.item()) == 0x8 and (out[-1] == 0).all()
    else:
        out = lmh.project_q4(x[idx.clamp(max=T - 1).long()], table, dev_status=status)
        assert int(status.item()) == 0
    assert torch.equal(out[:-1], few[idx[:-1].long()])
