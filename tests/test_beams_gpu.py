"""Beam selection from logits and from top-k lists against scores in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


def _candidates(logits, scores, beams, mask=None, finished=None, pad=0):
    """Per group: (scores in 64 bits, beams, tokens) of all continuations, best first, ties by beam and token."""
    z = logits.double().cpu()
    z = torch.where(torch.isnan(z), -INF, z)
    rows, V = z.shape
    plus = (z == INF).any(1, keepdim=True)
    z = torch.where(plus, torch.where(z == INF, 0.0, -INF), z)
    m = z.amax(1, keepdim=True)
    lp = (z - m) - torch.log(torch.exp(z - m).sum(1, keepdim=True))  # (m + log ... would lose the log at 3e38)
    if mask is not None:
        v = torch.arange(V)
        lp = torch.where((mask.cpu()[:, v // 32] >> (v % 32).int()) & 1 != 0, lp, -INF)
    s = scores.double().cpu()
    score = s[:, None] + lp
    token = torch.arange(V).expand(rows, V).clone()
    if finished is not None:
        for r in finished.cpu().nonzero().flatten().tolist():
            score[r] = -INF
            score[r, 0] = s[r]
            token[r, 0] = pad
    score = torch.where(torch.isfinite(s)[:, None] & (score.float() > -INF), score, -INF)
    out = []
    for g in range(rows // beams):
        flat = score[g * beams:(g + 1) * beams].flatten()
        order = flat.sort(descending=True, stable=True).indices
        order = order[flat[order] > -INF]
        out.append((flat[order], order // V + g * beams, token[g * beams:(g + 1) * beams].flatten()[order], flat, V))
    return out


def _tol(V, score):
    """A score's fp32 rounding, and the log-sum-exp's error: 2^-22 a term from the exponential, half a step for each
    of its argument's two roundings (log V at most in the mean), 32 roundings of a sum of positive terms."""
    return 2.0 ** -24 * score.abs() + 2.0 ** -22 + math.log(max(V, 2)) * 2.0 ** -23 + 32 * 2.0 ** -24


def _check(o, cands, beams, k, pad=0, finished=None, keep=False):
    """Scores in order and within the tolerance; every continuation is one, once, and has its score; exact
    equality of the choice where no two scores are nearer than the tolerance."""
    for g, (best, parent, token, flat, V) in enumerate(cands):
        s, p, t = (o[n][g].cpu() for n in ("scores", "parents", "tokens"))
        if keep:
            _check_slots(s, p, t, g, beams)
            order = s.double().sort(descending=True, stable=True).indices
            s, p, t = s[order], p[order], t[order]
        n = min(k, len(best))
        assert (p[n:] == -1).all() and (t[n:] == -1).all() and (s[n:] == -INF).all()
        s, p, t = s[:n], p[:n], t[:n]
        tol = _tol(V, best[:n])
        assert ((s.double() - best[:n]).abs() <= tol).all(), (g, s, best[:n])
        local = p.long() - g * beams
        ended = torch.zeros(n, dtype=torch.bool) if finished is None else finished.cpu()[p.long()].bool()
        at = local * V + torch.where(ended, 0, t.long())
        assert len(set(at.tolist())) == n and (local >= 0).all() and (local < beams).all()
        assert (t[ended] == pad).all()
        assert ((flat[at] - s.double()).abs() <= tol).all()
        near = (best[:n + 1].diff().abs() <= 2 * _tol(V, best[1:n + 1])) & (best[:n + 1].diff() != 0)
        if not near.any() and not keep:
            assert torch.equal(p.long(), parent[:n]) and torch.equal(t.long(), token[:n]), g


def _check_slots(s, p, t, g, beams):
    """A parent's best continuation stands in its place; the others fill the places left over, best first."""
    base = g * beams
    real = [r for r in range(beams) if p[r] >= 0]
    for r in real:
        assert p[int(p[r]) - base] == p[r]  # the parent's own place holds one of its children
    firsts = {int(p[r]) - base for r in real}
    for r in firsts:
        assert all(s[r] >= s[q] for q in real if p[q] == p[r])
    rest = [float(s[r]) for r in range(beams) if r not in firsts]
    assert rest == sorted(rest, reverse=True)


def _logits(rows, V, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    z = 2 * torch.randn(rows, V, generator=g, device="cuda")
    top = torch.randint(0, V, (rows, 12), generator=g, device="cuda")
    z.scatter_(1, top, 6 + 3 * torch.randn(rows, 12, generator=g, device="cuda"))
    return z.to(dtype), -3 - 3 * torch.rand(rows, generator=g, device="cuda")


def _mask(rows, V, share, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    words = (V + 31) // 32
    bits = (torch.rand(rows, words * 32, generator=g, device="cuda") < share).view(rows, words, 32).long()
    packed = (bits << torch.arange(32, device="cuda")).sum(-1)
    return (packed - ((packed >> 31) << 32)).int()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("groups,beams,k,V", [(1, 1, 1, 1), (1, 4, 8, 5), (3, 2, 4, 65), (2, 4, 8, 4100),
                                              (5, 3, 3, 1000), (2, 8, 16, 20001), (1, 32, 64, 8192), (2, 128, 128, 513),
                                              (1, 5, 128, 130), (1, 4, 8, 151936)])
def test_against_64_bits(lmh, groups, beams, k, V, dtype):
    z, s = _logits(groups * beams, V, dtype, V + beams)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = lmh.beam_select(z, s, beams, k=k, dev_status=st)
    assert int(st.item()) == 0
    _check(o, _candidates(z, s, beams), beams, k)


@pytest.mark.parametrize("share", [0.0, 1e-3, 0.05, 1.0])
@pytest.mark.parametrize("V", [97, 4100, 30000])
def test_masks(lmh, V, share):
    from top_reduction_gb300 import lmh as L
    z, s = _logits(12, V, torch.float32, V)
    m = _mask(12, V, share, 5)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cands = _candidates(z, s, 4, mask=m)
    o = lmh.beam_select(z, s, 4, k=8, mask=m, dev_status=st)
    _check(o, cands, 4, 8)
    assert int(st.item()) == (L.DS_NO_ALLOWED_TOKEN if any(len(c[0]) == 0 for c in cands) else 0)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("beams", [1, 2, 4, 7, 32, 128])
def test_ended_beams_and_slots(lmh, beams, keep):
    rows = 3 * beams
    z, s = _logits(rows, 3001, torch.bfloat16, beams)
    done = torch.arange(rows, device="cuda") % 3 == 1
    z[done] = float("nan")  # not read
    o = lmh.beam_select(z, s, beams, finished=done, pad_id=9, keep_slots=keep)
    _check(o, _candidates(z, s, beams, finished=done, pad=9), beams, beams, pad=9, finished=done, keep=keep)
    if keep:  # the same set as without slots
        plain = lmh.beam_select(z, s, beams, finished=done, pad_id=9)
        for g in range(3):
            a, b = ({(int(p), int(t)) for p, t in zip(q["parents"][g], q["tokens"][g])} for q in (o, plain))
            assert a == b


def test_all_beams_ended(lmh):
    s = torch.tensor([-3.0, -1.0, -2.0, -INF], device="cuda")
    z = torch.zeros(4, 100, device="cuda")
    o = lmh.beam_select(z, s, 4, finished=torch.ones(4, dtype=torch.uint8, device="cuda"), pad_id=-5)
    assert o["parents"].tolist() == [[1, 2, 0, -1]] and o["tokens"].tolist() == [[-5, -5, -5, -1]]
    assert o["scores"].tolist() == [[-1.0, -2.0, -3.0, -INF]]


def test_the_first_step(lmh):
    """All beams alike, all but the first with a score of -inf: the first row's best tokens."""
    z = _logits(1, 5000, torch.float32, 3)[0].expand(4, 5000).contiguous()
    s = torch.tensor([0.0, -INF, -INF, float("nan")], device="cuda")
    o = lmh.beam_select(z, s, 4)
    assert o["parents"].tolist() == [[0] * 4]
    assert o["tokens"][0].tolist() == z[0].double().sort(descending=True, stable=True).indices[:4].tolist()


@pytest.mark.parametrize("k,V", [(8, 70), (16, 4096), (128, 20000), (8, 151936)])
def test_ties_go_by_beam_then_token(lmh, k, V):
    """Rows alike, all logits equal: the fast path's lists overflow, and the order is the tokens'."""
    z = torch.zeros(6, V, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(6, device="cuda")
    s[4] = 0.25  # the second group's second beam leads
    o = lmh.beam_select(z, s, 3, k=k)
    n = min(k, V)
    assert o["parents"][0].tolist() == [i // V for i in range(k)]
    assert o["tokens"][0].tolist() == [i % V for i in range(k)]
    assert o["parents"][1, :n].tolist() == [4] * n and o["tokens"][1, :n].tolist() == list(range(n))
    z[:, 1::2] = -3.0e38  # masked by a lowest value, in places
    o = lmh.beam_select(z, s, 3, k=k)
    want = [(b, t) for b in range(3) for t in range(0, V, 2)][:k]
    assert list(zip(o["parents"][0].tolist(), o["tokens"][0].tolist()))[:len(want)] == want


@pytest.mark.parametrize("fill", [-INF, torch.finfo(torch.float32).min, torch.finfo(torch.bfloat16).min])
def test_few_tokens_above_the_lowest_value(lmh, fill):
    """Masked in the logits themselves: fewer tokens stand out than are asked for."""
    z = torch.full((4, 9000), fill, device="cuda")
    z[0, 17] = 2.0
    z[2, 8999] = 1.0
    z[2, 63] = 1.5
    s = torch.tensor([-1.0, -2.0, -0.5, -9.0], device="cuda")
    o = lmh.beam_select(z, s, 4, k=8)
    _check(o, _candidates(z, s, 4), 4, 8)


def test_infinities_and_nan(lmh):
    z, s = _logits(8, 3000, torch.float32, 1)
    z[0, 5] = z[0, 2000] = INF
    z[1] = -INF
    z[2, ::7] = float("nan")
    z[3] = float("nan")
    z[5, 100:200] = INF
    z[6, 64:128] = -INF
    s[4] = INF
    o = lmh.beam_select(z, s, 4, k=8)
    s[4] = -INF  # (a score that is not finite: none)
    _check(o, _candidates(z, s, 4), 4, 8)


def test_scores_far_apart_and_large(lmh):
    z, s = _logits(8, 2000, torch.float32, 2)
    s[1], s[2], s[5] = -1e30, -3.4e38, 1e6
    z[3] *= 1e20
    z[6] -= 1e4
    o = lmh.beam_select(z, s, 4, k=8)
    _check(o, _candidates(z, s, 4), 4, 8)


def test_strides_alignment_and_streams(lmh):
    z, s = _logits(8, 4099, torch.bfloat16, 9)
    want = lmh.beam_select(z, s, 4, k=8)
    wide = torch.full((8, 4112), INF, dtype=torch.bfloat16, device="cuda")
    for at in (0, 1, 8):
        wide.fill_(INF)
        wide[:, at:at + 4099] = z
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        got = lmh.beam_select(wide[:, at:at + 4099], s, 4, k=8, stream=st)
        st.synchronize()
        # (a row's terms are summed in another order where it begins elsewhere: scores agree to twice the tolerance)
        assert torch.equal(got["parents"], want["parents"]) and torch.equal(got["tokens"], want["tokens"])
        a, b = (o["scores"].double().cpu() for o in (got, want))
        assert ((a - b).abs() <= 2 * _tol(4099, b)).all()


@pytest.mark.parametrize("groups,beams,n,k", [(1, 1, 1, 1), (3, 4, 20, 8), (2, 8, 5, 16), (2, 128, 128, 128), (4, 3, 7, 3)])
def test_lists(lmh, groups, beams, n, k):
    rows = groups * beams
    z, s = _logits(rows, max(n, 3000), torch.float32, n)
    top = lmh.logprobs_from_logits(z, k_max=n)
    row_k = torch.arange(rows, device="cuda") % (n + 1)
    cut = torch.arange(n, device="cuda")[None] >= row_k[:, None]
    ids, lp = top["topk_ids"].masked_fill(cut, -1), top["topk_logprobs"].masked_fill(cut, -INF)
    done = torch.arange(rows, device="cuda") % 5 == 4
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = lmh.beam_select_lists(ids, lp, s, beams, k=k, finished=done, pad_id=77, dev_status=st)
    score = torch.where(ids < 0, -INF, s.double()[:, None] + lp.double())
    first = torch.arange(n, device="cuda")[None] == 0
    score = torch.where(done[:, None], torch.where(first, s.double()[:, None], -INF), score)
    ids = torch.where(done[:, None], 77, ids)
    for g in range(groups):
        flat = score[g * beams:(g + 1) * beams].flatten().cpu()
        order = flat.sort(descending=True, stable=True).indices
        order = order[flat[order] > -INF][:k]
        want_p, want_t = order // n + g * beams, ids[g * beams:(g + 1) * beams].flatten().cpu()[order]
        m = len(order)
        assert o["parents"][g, :m].tolist() == want_p.tolist() and o["tokens"][g, :m].tolist() == want_t.tolist()
        assert torch.equal(o["scores"][g, :m].cpu(), flat[order].float())
        assert (o["parents"][g, m:] == -1).all() and (o["scores"][g, m:] == -INF).all()


def test_lists_agree_with_logits(lmh):
    z, s = _logits(32, 20000, torch.float32, 4)
    top = lmh.logprobs_from_logits(z, k_max=8)
    a = lmh.beam_select(z, s, 4, k=8)
    b = lmh.beam_select_lists(top["topk_ids"], top["topk_logprobs"], s, 4, k=8)
    for g, c in enumerate(_candidates(z, s, 4)):
        near = c[0][:9].diff().abs().min()
        assert near > 1e-4  # (otherwise the rounding of the lists' logprobs may change places)
    assert torch.equal(a["parents"], b["parents"]) and torch.equal(a["tokens"], b["tokens"])
    assert torch.allclose(a["scores"], b["scores"], rtol=0, atol=4e-6)


def test_list_entries_that_are_none(lmh):
    ids = torch.tensor([[5, -1, 7, 8], [9, 9, 3, 2]], dtype=torch.int32, device="cuda")
    lp = torch.tensor([[-1.0, -0.5, float("nan"), INF], [-1.0, -1.0, -INF, -4.0]], device="cuda")
    o = lmh.beam_select_lists(ids, lp, torch.zeros(2, device="cuda"), 2, k=6)
    assert o["parents"].tolist() == [[0, 1, 1, 1, -1, -1]] and o["tokens"].tolist() == [[5, 9, 9, 2, -1, -1]]


def test_graph_replays_share_a_workspace(lmh):
    zs = [_logits(12, 9001, torch.bfloat16, i) for i in range(4)]
    want = [lmh.beam_select(z, s, 4, k=8) for z, s in zs]
    ws = torch.empty(max(lmh.beam_workspace_bytes(12, 4, 9001), 256), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [lmh.beam_select(z, s, 4, k=8, workspace=ws) for z, s in zs]
    for _ in range(3):
        ws.random_(0, 256)
        for o in got:
            o["scores"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("kw,what", [
    (dict(beams=3), "whole groups"), (dict(beams=0), "whole groups"), (dict(scores=None), "scores is required"),
    (dict(finished=torch.zeros(3)), "8 entries"), (dict(mask=torch.zeros(8, 4)), "mask must be"),
    (dict(out="long"), "parents must be"), (dict(workspace="small"), "workspace must be")])
def test_binding_refusals(lmh, kw, what):
    z, s = _logits(8, 500, torch.float32, 1)
    if kw.get("out") == "long":
        kw = dict(out={"scores": torch.zeros(2, 4, device="cuda"), "tokens": torch.zeros(2, 4, device="cuda").int(),
                       "parents": torch.zeros(2, 4, device="cuda").long()})
    if kw.get("workspace") == "small":
        kw = dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    a = dict(dict(logits=z, scores=s, beams=4), **kw)
    with pytest.raises(ValueError, match=what):
        lmh.beam_select(**a)
