"""Beam search of several requests, each with adapters of its own, around a 4-bit embedding and head.

    python examples/beam_decode.py [--vocab 151936] [--hidden 1024] [--groups 8] [--beams 4] [--steps 16]

A step embeds the beams' last tokens (lookup_q4), runs a body (here one recurrent layer of random
weights, in the model's place) whose projection and whose head carry the requests' low-rank adapters
(add_adapters, beside a matrix product and in place on project_q4's logits), takes every request's best
continuations over its beams and the vocabulary (beam_select, survivors in their places) and lets the
beams' states, the token histories as far as they are in use, follow their parents in place
(reorder_rows).  Everything stays at one address, so the step is captured once in a CUDA graph and a
replay is the whole step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Model:
    """One recurrent layer of random weights between a 4-bit table's two ends, with adapters per request."""

    def __init__(self, vocab, hidden, adapters, rank, seed=0, device="cuda"):
        import top_reduction_gb300 as lmh
        gen = torch.Generator(device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device=device)
        self.lmh, self.hidden, self.device = lmh, hidden, device
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.table = lmh.quantize_q4((4 * randn(vocab, hidden) * hidden ** -0.5).to(torch.bfloat16), group=64)
        self.body = (randn(hidden, hidden) * hidden ** -0.5).to(torch.bfloat16)

        def table(n):
            return lmh.AdapterTable((randn(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16),
                                    (randn(adapters, n, rank) * 0.2).to(torch.bfloat16),
                                    scales=torch.full((adapters,), 0.5, device=device))
        self.body_adapters, self.head_adapters = table(hidden), table(vocab)

    def step(self, ids, state, adapter_idx):
        """The logits of the next tokens; `state` moves on in place."""
        lmh = self.lmh
        x = lmh.lookup_q4(ids, self.table, scale=self.hidden ** 0.5 / 4, dev_status=self.status)
        y = lmh.add_adapters(x, self.body_adapters, adapter_idx, x @ self.body, dev_status=self.status)
        state.copy_(0.5 * state + torch.nn.functional.silu(y))
        logits = lmh.project_q4(state, self.table, dev_status=self.status)
        return lmh.add_adapters(state, self.head_adapters, adapter_idx, logits, out=logits, dev_status=self.status)


def run(vocab=151936, hidden=1024, groups=8, beams=4, steps=16, adapters=3, rank=16, eos=2, seed=0, device="cuda"):
    """Returns (tokens int32 [groups * beams, steps], lengths, scores, us per step, the model, the adapters' indices)."""
    import top_reduction_gb300 as lmh
    model = Model(vocab, hidden, adapters, rank, seed, device)
    rows = groups * beams
    # request g uses adapter g, and every (adapters + 1)-th one none
    adapter_idx = ((torch.arange(groups, device=device) + 1) % (adapters + 1) - 1).int().repeat_interleave(beams)
    ids = torch.ones(rows, dtype=torch.int32, device=device)
    state = torch.zeros(rows, hidden, dtype=torch.bfloat16, device=device)
    history = torch.zeros(rows, steps, dtype=torch.int32, device=device)
    lengths = torch.zeros(rows, dtype=torch.int32, device=device)
    finished = torch.zeros(rows, dtype=torch.uint8, device=device)
    scores = torch.full((groups, beams), -float("inf"), device=device)
    scores[:, 0] = 0.0  # at first a request's beams are one
    first = [t.clone() for t in (ids, state, history, lengths, finished, scores)]
    states = lmh.RowStates([history, state, finished], length_dims=[1, None, None])

    def step():
        logits = model.step(ids, state, adapter_idx)
        o = lmh.beam_select(logits, scores, beams, finished=finished, pad_id=eos, keep_slots=True, dev_status=model.status)
        lmh.reorder_rows(states, o["parents"], beams, lengths=lengths, dev_status=model.status)
        token = o["tokens"].view(rows)
        history.scatter_(1, lengths[:, None].long(), token[:, None])
        finished.copy_(finished | (token == eos))
        lengths.add_(1)
        ids.copy_(token)
        scores.copy_(o["scores"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (warm-up: libraries choose their algorithms outside the capture)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, f in zip((ids, state, history, lengths, finished, scores), first):
        t.copy_(f)

    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if int(model.status.item()):
        raise RuntimeError("device status %#x" % int(model.status.item()))
    return history, lengths, scores, begin.elapsed_time(end) * 1e3 / max(steps, 1), model, adapter_idx


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=151936)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    tokens, _, scores, us, _, _ = run(a.vocab, a.hidden, a.groups, a.beams, a.steps)
    for g in range(min(a.groups, 2)):
        for b in scores[g].argsort(descending=True).tolist():
            print("request %d, score %8.3f: %s" % (g, float(scores[g, b]), tokens[g * a.beams + b].tolist()))
    print("%d requests of %d beams, %d x %d table: %.1f us a step" % (a.groups, a.beams, a.hidden, a.vocab, us))


if __name__ == "__main__":
    main()
