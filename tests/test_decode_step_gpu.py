"""The 4-bit table's operators and the filtered draw together, and their bounded waits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("vocab,hidden,rows,steps", [(5003, 256, 7, 3), (20000, 512, 20, 2), (1000, 128, 1, 1)])
def test_example(lmh, vocab, hidden, rows, steps):
    import q4_decode
    ids, model, drawn, _ = q4_decode.run(vocab, hidden, rows, steps)
    again = q4_decode.run(vocab, hidden, rows, steps)
    assert ids.shape == (rows, steps + 1) and int(ids.min()) >= 0 and int(ids.max()) < vocab
    for a, b in zip((ids, model, drawn), again):
        assert torch.equal(a, b)
    greedy = torch.arange(rows) % 3 == 0
    assert (drawn.cpu()[greedy] == 0).all()          # the only token of its distribution
    assert (model <= 1e-5).all() and (drawn <= 1e-6).all()


def _tables(lmh, rows, V, H):
    gen = torch.Generator("cuda").manual_seed(rows)
    W = torch.randn(V, H, generator=gen, device="cuda").to(torch.bfloat16)
    x = torch.randn(rows, H, generator=gen, device="cuda").to(torch.bfloat16)
    return lmh.quantize_q4(W, 64), x, torch.rand(rows, generator=gen, device="cuda")


@pytest.mark.parametrize("rows,V,H", [(1, 20000, 1024), (12, 20000, 1024), (20, 20000, 1024), (8, 20000, 16384),
                                      (32, 300000, 2560)])
def test_projection_wait_runs_out_then_recovers(lmh, rows, V, H):
    """With a limit of 1 ns a call reports that a wait ran out, or is right; the next call is right.
    (A small table's boxes are there before anybody waits; the large one does not fit in L2.)"""
    from top_reduction_gb300 import lmh as L
    table, x, _ = _tables(lmh, rows, V, H)
    want = lmh.project_q4(x, table)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    try:
        L.debug_set_wait_limit(1)
        got = lmh.project_q4(x, table, dev_status=st)
        torch.cuda.synchronize()  # the grid finished
    finally:
        L.debug_set_wait_limit(0)
    assert int(st.item()) == L.DS_TIMEOUT or (int(st.item()) == 0 and V < 300000 and torch.equal(got, want))
    st.zero_()
    assert torch.equal(lmh.project_q4(x, table, dev_status=st), want)
    assert int(st.item()) == 0


def test_sampling_wait_runs_out_then_recovers(lmh):
    from top_reduction_gb300 import lmh as L
    table, x, u = _tables(lmh, 16, 100000, 128)
    logits = lmh.project_q4(x, table)
    p = torch.full((16,), 0.9, device="cuda")
    want = lmh.sample_from_logits(logits, u, top_p=p)["sampled_ids"].clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    try:
        L.debug_set_wait_limit(1)
        lmh.sample_from_logits(logits, u, top_p=p, dev_status=st)
        torch.cuda.synchronize()
    finally:
        L.debug_set_wait_limit(0)
    assert int(st.item()) & L.DS_TIMEOUT
    st.zero_()
    assert torch.equal(lmh.sample_from_logits(logits, u, top_p=p, dev_status=st)["sampled_ids"], want)
    assert int(st.item()) == 0


@pytest.mark.parametrize("rows,V", [(4, 151936), (32, 50000), (64, 8000)])
def test_logprobs_follow_the_projection_and_the_draw(lmh, rows, V):
    """logprobs_from_logits reads its first chunks and the selected ids ahead of the stream's order,
    unless the kernel before has to end first: it does after project_q4 and after a draw."""
    table, _, _ = _tables(lmh, 1, V, 256)
    gen = torch.Generator("cuda").manual_seed(V)
    xs = [torch.randn(rows, 256, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(12)]
    us = torch.rand(12, rows, generator=gen, device="cuda")
    p = torch.full((rows,), 0.95, device="cuda")
    z = torch.empty(rows, V, device="cuda")
    draw = {"sampled_ids": torch.empty(rows, dtype=torch.int32, device="cuda"),
            "sampled_logprob": torch.empty(rows, device="cuda")}

    def steps(sync):
        got = []
        for x, u in zip(xs, us):
            lmh.project_q4(x, table, out=z)
            if sync:
                torch.cuda.synchronize()
            lse = lmh.logprobs_from_logits(z)["lse"]
            lmh.sample_from_logits(z, u, top_p=p, out=draw)
            if sync:
                torch.cuda.synchronize()
            sel = lmh.logprobs_from_logits(z, sel=draw["sampled_ids"])["sel_logprob"]
            got.append((lse.clone(), sel.clone()))
        if sync:
            torch.cuda.synchronize()
        return got
    want = steps(True)
    graph = torch.cuda.CUDAGraph()  # (a graph's kernels follow one another at once)
    with torch.cuda.graph(graph):
        got = steps(False)
    for replay in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a[0], b[0]), "projection, step %d" % i
            assert torch.equal(a[1], b[1]), "draw, step %d" % i
