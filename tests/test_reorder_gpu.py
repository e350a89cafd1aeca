"""States that follow their rows (lmh_reorder_rows): copies, so every byte is compared."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _parents(groups, beams, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "self":
        p = torch.arange(beams).expand(groups, beams).clone()
    elif kind == "swap":  # every row is a source and replaced
        p = torch.stack([torch.randperm(beams, generator=g) for _ in range(groups)])
    elif kind == "one":
        p = torch.full((groups, beams), beams - 1)
    else:
        p = torch.randint(0, beams, (groups, beams), generator=g)
    p = p + beams * torch.arange(groups)[:, None]
    if kind == "some":
        p[torch.rand(groups, beams, generator=g) < 0.3] = -1
    return p.int().cuda()


def _want(t, old, dim, along, parents, lengths):
    p = parents.flatten().long()
    p = torch.where(p < 0, torch.arange(len(p), device="cuda"), p)
    new = t.index_select(dim, p)
    if along is None or lengths is None:
        return new
    at = [1] * t.dim()
    at[along] = t.shape[along]
    rows = [1] * t.dim()
    rows[dim] = len(p)
    return torch.where(torch.arange(t.shape[along], device="cuda").view(at) < lengths.long()[p].view(rows), new, old)


def _states(rows, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def whole(dtype, *shape):
        return torch.randint(-2 ** 31, 2 ** 31 - 1, shape, generator=g, device="cuda").to(dtype)
    cache = whole(torch.int16, 2, 2, rows, 3, 40, 24)
    return [(whole(torch.int32, rows, 77), 0, 1), (whole(torch.uint8, rows, 5), 0, None), (whole(torch.int64, rows), 0, None),
            (whole(torch.int32, rows, 9000), 0, None), (whole(torch.int16, 3, rows, 1001), 1, 2),
            (cache, 2, 4), (whole(torch.int16, 2, 2, rows, 3, 40, 24)[:, 1, :, :, :33], 1, 3),
            (whole(torch.int32, rows, 6, 8)[:, ::2], 0, None), (whole(torch.uint8, 130, rows).t(), 0, None)]


@pytest.mark.parametrize("kind", ["self", "swap", "one", "any", "some"])
@pytest.mark.parametrize("groups,beams", [(1, 1), (1, 4), (5, 3), (2, 33), (1, 128), (70, 2)])
def test_in_place_and_out_of_place(lmh, groups, beams, kind):
    rows = groups * beams
    p = _parents(groups, beams, rows, kind)
    g = torch.Generator("cuda").manual_seed(1)
    lengths = torch.randint(-2, 50, (rows,), generator=g, device="cuda", dtype=torch.int32)
    for use in (None, lengths):
        made = _states(rows, beams)
        tensors, dims, along = [list(v) for v in zip(*made)]
        outs = [torch.full_like(t, 7) if t.is_contiguous() else t.clone() * 0 for t in tensors]
        want = [_want(t, o, d, a, p, use) for t, o, d, a in zip(tensors, outs, dims, along)]
        before = [t.clone() for t in tensors]
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = lmh.reorder_rows(lmh.RowStates(tensors, dims, along, outs), p, beams, lengths=use, dev_status=st)
        for t, b, o, w in zip(tensors, before, got, want):
            assert torch.equal(t, b) and torch.equal(o, w)
        want = [_want(t, t, d, a, p, use) for t, d, a in zip(tensors, dims, along)]
        lmh.reorder_rows(lmh.RowStates(tensors, dims, along), p, beams, lengths=use, dev_status=st)
        for t, w in zip(tensors, want):
            assert torch.equal(t, w)
        assert int(st.item()) == 0


@pytest.mark.parametrize("kind", ["swap", "one", "any", "some"])
@pytest.mark.parametrize("groups,beams", [(1, 1), (3, 4), (5, 3), (1, 33), (1, 128), (40, 2)])
def test_large_states(lmh, groups, beams, kind):
    """States that move by bulk copies: positions of 4 and 48 bytes, chunks of odd multiples of 16 bytes, lengths that
    end inside a slice, before the first position and behind the last."""
    rows = groups * beams
    p = _parents(groups, beams, rows + 1, kind)
    g = torch.Generator("cuda").manual_seed(2)
    T = (24 << 20) // (4 * rows) // 4 * 4
    lengths = torch.randint(-2, T + T // 4, (rows,), generator=g, device="cuda", dtype=torch.int32)
    t = (24 << 20) // (48 * 12 * rows) + 1
    shorter = torch.clamp(lengths * t // T, max=t + 1)
    for tensors, dims, along, lens in (
            ([torch.randint(-99, 99, (rows, T), generator=g, device="cuda", dtype=torch.int32)], [0], [1], lengths),
            ([torch.randint(-99, 99, (2, 2, rows, 3, t, 24), generator=g, device="cuda", dtype=torch.int16),
              torch.randint(-99, 99, (3, rows, 4 * t, 8), generator=g, device="cuda", dtype=torch.int16)[:, :, 1:]],
             [2, 1], [4, None], shorter)):
        for use in (None, lens):
            first = [x.clone() for x in tensors]
            outs = [torch.full_like(x, 7) for x in first]
            want = [_want(x, o, d, a, p, use) for x, o, d, a in zip(first, outs, dims, along)]
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = lmh.reorder_rows(lmh.RowStates(tensors, dims, along, outs), p, beams, lengths=use, dev_status=st)
            assert all(torch.equal(o, w) for o, w in zip(got, want))
            want = [_want(x, x, d, a, p, use) for x, d, a in zip(first, dims, along)]
            lmh.reorder_rows(lmh.RowStates(tensors, dims, along), p, beams, lengths=use, dev_status=st)
            assert all(torch.equal(x, w) for x, w in zip(tensors, want))
            assert int(st.item()) == 0


def test_neighbours_are_left_alone(lmh):
    """Views in larger tensors: what lies between the rows and behind the positions stays."""
    whole = torch.arange(2 * 8 * 64, dtype=torch.int32, device="cuda").view(2, 8, 64)
    p = torch.tensor([[3, 3, 0, 1]], dtype=torch.int32, device="cuda")
    view = whole[:, 2:6, 5:50]
    want = whole.clone()
    want[:, 2:6, 5:50] = want[:, 2:6, 5:50][:, [3, 3, 0, 1]]
    lmh.reorder_rows(lmh.RowStates([view], dims=1), p, 4)
    assert torch.equal(whole, want)


def test_bad_parents(lmh):
    from top_reduction_gb300 import lmh as L
    t = torch.arange(8, device="cuda", dtype=torch.int32)[:, None].repeat(1, 9)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = torch.tensor([1, 4, 2 ** 30, -2, 5, 5, 3, 8], dtype=torch.int32, device="cuda")  # groups of four
    lmh.reorder_rows([t], p, 4, dev_status=st)
    assert t[:, 0].tolist() == [1, 1, 2, 3, 5, 5, 6, 7] and int(st.item()) == L.DS_ROW_IDX_OUT_OF_RANGE


def test_many_states(lmh):
    """More states than one launch takes, an empty one among them."""
    p = _parents(3, 4, 2, "any")
    tensors = [torch.randint(0, 99, (12, 3 + i), device="cuda") for i in range(60)] + [torch.zeros(12, 0, device="cuda")]
    want = [t[p.flatten().long()] for t in tensors]
    for t, w in zip(lmh.reorder_rows(tensors, p, 4), want):
        assert torch.equal(t, w)


def test_large_offsets(lmh):
    """Rows whose bytes begin beyond 2^32."""
    t = torch.zeros(4, 1 << 29, dtype=torch.int32, device="cuda")  # 2 GiB a row
    t[:, -1] = torch.arange(4, device="cuda", dtype=torch.int32) + 1
    t[:, 0] = 10 * t[:, -1]
    lmh.reorder_rows([t], torch.tensor([3, 1, 2, 0], dtype=torch.int32, device="cuda"), 4)
    assert t[:, -1].tolist() == [4, 2, 3, 1] and t[:, 0].tolist() == [40, 20, 30, 10]


def test_streams_and_graph(lmh):
    t = torch.randint(0, 1000, (3, 8, 500), device="cuda")
    p = torch.tensor([1, 2, 3, 0, 7, 7, 5, 4], dtype=torch.int32, device="cuda")
    states = lmh.RowStates([t], dims=1)
    first = t.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lmh.reorder_rows(states, p, 4, stream=st)
    st.synchronize()
    assert torch.equal(t, first[:, p.long()])
    t.copy_(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            lmh.reorder_rows(states, p, 4)
    want = first
    for _ in range(3):
        want = want[:, p.long()]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(t, want)
