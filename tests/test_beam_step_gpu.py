"""Adapters, beam selection and reordering together, as a captured decode step; calls that follow one another at
once; bounded waits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("vocab,hidden,groups,beams,steps,eos", [(5003, 128, 3, 4, 5, 2), (2000, 64, 1, 1, 4, 7),
                                                                 (20000, 256, 5, 7, 3, 2), (300, 64, 4, 3, 12, 2)])
def test_example_scores_are_its_histories(lmh, vocab, hidden, groups, beams, steps, eos):
    """Every beam's history, fed back row by row without any reordering, has the beam's score: a state that had not
    followed its parent would give another.  The log-probabilities are those of logprobs_from_logits, each within 1e-5;
    the scores are rounded to fp32 once a step."""
    import beam_decode
    tokens, lengths, scores, _, model, idx = beam_decode.run(vocab, hidden, groups, beams, steps, eos=eos)
    again = beam_decode.run(vocab, hidden, groups, beams, steps, eos=eos)
    assert torch.equal(tokens, again[0]) and torch.equal(scores, again[2])
    rows = groups * beams
    assert (lengths == steps).all() and int(tokens.min()) >= 0 and int(tokens.max()) < vocab
    for g in range(groups):
        assert len({tuple(t) for t in tokens[g * beams:(g + 1) * beams].tolist()}) == beams
    ids = torch.ones(rows, dtype=torch.int32, device="cuda")
    state = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    total = torch.zeros(rows, dtype=torch.float64, device="cuda")
    live = torch.ones(rows, dtype=torch.bool, device="cuda")
    for s in range(steps):
        logits = model.step(ids, state, idx)
        ids = tokens[:, s].contiguous()
        lp = model.lmh.logprobs_from_logits(logits, sel=ids)["sel_logprob"].double()
        total += torch.where(live, lp, 0.0)
        assert (live | (ids == eos)).all()  # an ended beam goes on with the padding token
        live &= ids != eos
    off = steps * (1e-5 + 2.0 ** -24 * scores.abs().max())
    assert ((total - scores.view(-1).double()).abs() <= off).all(), (total, scores)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("rows,H,V,R", [(8, 128, 5000, 8), (32, 256, 50001, 16), (300, 64, 2048, 32)])
def test_steps_that_follow_at_once(lmh, rows, H, V, R):
    """Projection, adapters in place, selection and reordering, step after step in a graph with new inputs at every
    replay, against the same calls one by one: none reads what the one before it has not yet written."""
    beams, steps = 4, 6
    W = _randn(1, V, H).to(torch.bfloat16)
    table = lmh.quantize_q4(W, 64)
    ad = lmh.AdapterTable((_randn(2, 3, R, H) * H ** -0.5).to(torch.bfloat16), _randn(3, 3, V, R).to(torch.bfloat16))
    idx = (torch.arange(rows, device="cuda") % 4 - 1).int()
    x = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    scores = torch.empty(rows, device="cuda")
    hist = torch.empty(rows, 40, dtype=torch.int32, device="cuda")
    z = torch.empty(rows, V, device="cuda")
    out = {"scores": torch.empty(rows // beams, beams, device="cuda"),
           "parents": torch.empty(rows // beams, beams, dtype=torch.int32, device="cuda"),
           "tokens": torch.empty(rows // beams, beams, dtype=torch.int32, device="cuda")}
    states = lmh.RowStates([x, hist])

    def run(sync):
        got = []
        for s in range(steps):
            calls = (lambda: lmh.project_q4(x, table, out=z), lambda: lmh.add_adapters(x, ad, idx, z, out=z),
                     lambda: lmh.beam_select(z, scores, beams, out=out), lambda: lmh.reorder_rows(states, out["parents"], beams),
                     lambda: scores.copy_(out["scores"].view(-1)), lambda: hist[:, s].copy_(out["tokens"].view(-1)))
            for c in calls:
                c()
                if sync:
                    torch.cuda.synchronize()
            got += [out["tokens"].clone(), out["scores"].clone(), hist.clone(), x.clone()]
        return got

    def refill(seed):
        x.copy_(_randn(seed, rows, H))
        scores.copy_(-_randn(seed + 1, rows).abs())
        hist.zero_()
    refill(0)
    run(True)
    refill(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(False)
    for replay in range(1, 4):
        refill(10 * replay)
        want = [t.clone() for t in run(True)]
        refill(10 * replay)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), "replay %d, result %d" % (replay, i)


def test_two_streams_at_once(lmh):
    """Calls on two streams have workspaces of their own."""
    z = [_randn(i, 64, 30000) for i in range(2)]
    s = [-_randn(5 + i, 64).abs() for i in range(2)]
    x = [_randn(7 + i, 300, 256).to(torch.bfloat16) for i in range(2)]
    y = [_randn(9 + i, 300, 512) for i in range(2)]
    ad = lmh.AdapterTable(_randn(11, 4, 16, 256).to(torch.bfloat16), _randn(12, 4, 512, 16).to(torch.bfloat16))
    idx = [(torch.arange(300, device="cuda") * (3 + i) % 5 - 1).int() for i in range(2)]
    want = [(lmh.beam_select(z[i], s[i], 4)["scores"].clone(), lmh.add_adapters(x[i], ad, idx[i], y[i])) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [[], []]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                for _ in range(5):
                    got[i].append((lmh.beam_select(z[i], s[i], 4)["scores"], lmh.add_adapters(x[i], ad, idx[i], y[i])))
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in got[i]:
                assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])


def test_waits_run_out_then_recover(lmh):
    """With a limit of 1 ns a call reports that a wait ran out, or is right; the next call is right."""
    from top_reduction_gb300 import lmh as L
    z, s = _randn(1, 64, 200000), -_randn(2, 64).abs()
    want = lmh.beam_select(z, s, 4)
    big = torch.arange(8 << 20, device="cuda", dtype=torch.int32).view(8, 1 << 20)
    p = torch.tensor([1, 0, 3, 2, 4, 4, 4, 4], dtype=torch.int32, device="cuda")
    moved = big[p.long()]
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty_like(big)
    torch.cuda.synchronize()
    try:
        L.debug_set_wait_limit(1)
        lmh.beam_select(z, s, 4, dev_status=st[:1])
        lmh.reorder_rows(lmh.RowStates([big], outs=[out]), p, 4, dev_status=st[1:])
        torch.cuda.synchronize()
    finally:
        L.debug_set_wait_limit(0)
    assert all(v in (0, L.DS_TIMEOUT) for v in st.tolist()) and int(st[0]) == L.DS_TIMEOUT
    st.zero_()
    got = lmh.beam_select(z, s, 4, dev_status=st[:1])
    assert all(torch.equal(got[n], want[n]) for n in want)
    lmh.reorder_rows(lmh.RowStates([big], outs=[out]), p, 4, dev_status=st[1:])
    assert torch.equal(out, moved) and st.tolist() == [0, 0]


def test_first_calls_need_no_other_family(lmh):
    """A state is reordered, beams are chosen and adapters added as a process's first call."""
    import subprocess
    code = ("import torch, top_reduction_gb300 as l\n"
            "t = torch.arange(4, device='cuda').view(4, 1).float()\n"
            "l.reorder_rows([t], torch.tensor([1, 1, 0, 3], dtype=torch.int32, device='cuda'), 4)\n"
            "assert t.view(-1).tolist() == [1, 1, 0, 3]\n"
            "o = l.beam_select(torch.eye(4, 50, device='cuda'), torch.zeros(4, device='cuda'), 4)\n"
            "assert o['tokens'].tolist() == [[0, 1, 2, 3]]\n"
            "a = torch.ones(1, 8, 8, device='cuda', dtype=torch.bfloat16)\n"
            "y = l.add_adapters(a[0, :2], l.AdapterTable(a, a), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 8, device='cuda'))\n"
            "assert (y == 64).all()\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_on_one_stream(lmh):
    """Two host threads' kernels may come in turn on the stream that both call on."""
    import threading
    main = torch.cuda.current_stream()
    cases = []
    for i, rows in enumerate((300, 40)):
        ad = lmh.AdapterTable(_randn(20 + i, 4, 16, 256).to(torch.bfloat16), _randn(22 + i, 4, 520, 16).to(torch.bfloat16))
        c = dict(x=_randn(24 + i, rows, 256).to(torch.bfloat16), table=ad, y=_randn(26 + i, rows, 520),
                 adapter_idx=(torch.arange(rows, device="cuda") * 3 % 5 - 1).int())
        z, s = _randn(28 + i, 12, 9001), -_randn(30 + i, 12).abs()
        cases.append((c, z, s, lmh.add_adapters(**c), lmh.beam_select(z, s, 4)["scores"]))
    torch.cuda.synchronize()
    got = [[], []]

    def calls(i):
        c, z, s = cases[i][:3]
        with torch.cuda.stream(main):
            for _ in range(200):
                got[i].append((lmh.add_adapters(**c), lmh.beam_select(z, s, 4)["scores"]))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 200
        for a, b in got[i]:
            assert torch.equal(a, cases[i][3]) and torch.equal(b, cases[i][4])


def test_graphs_and_eager_calls_have_workspaces_of_their_own(lmh):
    """A graph captured without a workspace is replayed on one stream while eager calls run on another."""
    x, y = _randn(1, 300, 256).to(torch.bfloat16), _randn(2, 300, 512)
    ad = lmh.AdapterTable(_randn(3, 4, 16, 256).to(torch.bfloat16), _randn(4, 4, 512, 16).to(torch.bfloat16))
    idx = (torch.arange(300, device="cuda") * 3 % 5 - 1).int()
    z, s = _randn(5, 64, 30000), -_randn(6, 64).abs()
    other = (torch.arange(300, device="cuda") % 4).int()
    want = lmh.add_adapters(x, ad, idx, y), lmh.beam_select(z, s, 4)["scores"].clone()
    want2 = lmh.add_adapters(x, ad, other, y), lmh.beam_select(z + 1, s - 1, 4)["scores"].clone()
    z2, s2 = z + 1, s - 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = lmh.add_adapters(x, ad, idx, y), lmh.beam_select(z, s, 4)["scores"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.zero_()
        b.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        got = [(lmh.add_adapters(x, ad, other, y), lmh.beam_select(z2, s2, 4)["scores"]) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert all(torch.equal(p, want2[0]) and torch.equal(q, want2[1]) for p, q in got)


@pytest.mark.parametrize("rows", [3, 258])
def test_offsets_behind_32_bits(lmh, rows):
    """Rows, adapters and outputs further apart than 2^31 elements (few of them: 258 rows share a row of x)."""
    far = (1 << 30) + 8
    big = torch.zeros(3 * far, dtype=torch.bfloat16, device="cuda")
    H, N, R = 64, 520, 16
    down, up = _randn(1, 3, R, H).to(torch.bfloat16), _randn(2, 3, N, R).to(torch.bfloat16)
    x = _randn(3, 3, H).to(torch.bfloat16)
    at = 0  # each in its own part of the far rows
    views = []
    for t in (down, up, x):
        v = big.as_strided(t.shape, (far,) + t.stride()[1:], at)
        v.copy_(t)
        views.append(v)
        at += (t[0].numel() + 63) // 64 * 64
    row_idx = (torch.arange(rows, device="cuda") % 3).int()
    idx = ((torch.arange(rows, device="cuda") + 1) % 3).int()
    y = _randn(4, rows, N).to(torch.bfloat16)
    want = lmh.add_adapters(x, lmh.AdapterTable(down, up), idx, y, row_idx=row_idx)
    got = lmh.add_adapters(views[2], lmh.AdapterTable(views[0], views[1]), idx, y, row_idx=row_idx)
    assert torch.equal(got, want)
    if rows == 3:  # outputs and logits too
        out = big.as_strided((3, N), (far, 1), at)
        out.copy_(y)
        lmh.add_adapters(views[2], lmh.AdapterTable(views[0], views[1]), idx, out, row_idx=row_idx, out=out)
        assert torch.equal(out, want)
        s = torch.zeros(3, device="cuda")
        a, b = lmh.beam_select(out, s, 3), lmh.beam_select(want, s, 3)
        assert all(torch.equal(a[k], b[k]) for k in a)
