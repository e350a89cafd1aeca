"""Prompts and decode steps around a model body whose embedding and head are one 4-bit table.

    python examples/q4_decode.py [--vocab 151936] [--hidden 2560] [--rows 32] [--steps 16]

A batch of prompts is embedded (lookup_q4), run through a body (here a residual layer of random
weights, in the model's place), its last rows are picked (select_rows), projected through the same
table (project_q4) and sampled with the requests' temperature, top-k, top-p and min-p
(sample_from_logits).  The decode step that follows is captured once in a CUDA graph: its ids and
its uniform numbers stay at one address, so a replay is the whole step.  logprobs_from_logits gives
the drawn tokens' log-probabilities in the model's own distribution, next to those of the
distribution that was drawn from.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def run(vocab=151936, hidden=2560, rows=32, steps=16, group=64, seed=0, device="cuda"):
    """Returns (ids int32 [rows, steps + 1], model logprobs, drawn logprobs, us per decode step)."""
    import top_reduction_gb300 as lmh
    gen = torch.Generator(device).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    status = torch.zeros(1, dtype=torch.int32, device=device)
    table = lmh.quantize_q4((randn(vocab, hidden) * hidden ** -0.5).to(torch.bfloat16), group=group)
    body_w = (randn(hidden, hidden) * hidden ** -0.5).to(torch.bfloat16)

    def body(x):
        return x + torch.nn.functional.silu(x @ body_w)

    def embed(ids):
        return lmh.lookup_q4(ids, table, scale=hidden ** 0.5, dev_status=status)

    # what the requests ask for: every third one is greedy, the others use different filters
    i = torch.arange(rows, device=device)
    ask = {"temperature": torch.where(i % 3 == 0, 0.0, 0.8).float(),
           "top_k": torch.where(i % 3 == 1, 50, 0).int(),
           "top_p": torch.where(i % 3 == 2, 0.95, 1.0).float(),
           "min_p": torch.full((rows,), 0.02, device=device)}

    def draw(logits, u):
        o = lmh.sample_from_logits(logits, u, dev_status=status, **ask)
        model = lmh.logprobs_from_logits(logits, sel=o["sampled_ids"], k_max=0, dev_status=status)
        return o["sampled_ids"], model["sel_logprob"], o["sampled_logprob"]

    # prompts of different lengths, packed; only their last rows are projected
    lengths = 1 + i.cpu() % 7
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)]).int().to(device)
    prompt = torch.randint(0, vocab, (int(lengths.sum()),), generator=gen, device=device).int()
    row_idx, _ = lmh.select_rows(cu, 0, max_out_rows=rows, dev_status=status)
    logits = lmh.project_q4(body(embed(prompt)), table, row_idx=row_idx, rows=rows, dev_status=status)
    out = [[t.clone()] for t in draw(logits, torch.rand(rows, generator=gen, device=device))]

    ids, u = out[0][0].clone(), torch.empty(rows, device=device)

    def step():
        ids_next, model, drawn = draw(lmh.project_q4(body(embed(ids)), table, dev_status=status), u)
        ids.copy_(ids_next)
        return model, drawn

    uniforms = torch.rand(steps, rows, generator=gen, device=device)
    first = ids.clone()
    u.copy_(uniforms[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (warm-up: libraries choose their algorithms outside the capture)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model, drawn = step()
    ids.copy_(first)

    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for s in range(steps):
        u.copy_(uniforms[s])
        graph.replay()
        for kept, t in zip(out, (ids, model, drawn)):
            kept.append(t.clone())
    end.record()
    torch.cuda.synchronize()
    if int(status.item()):
        raise RuntimeError("device status %#x" % int(status.item()))
    ids_all, model_all, drawn_all = (torch.stack(t, 1) for t in out)
    return ids_all, model_all, drawn_all, begin.elapsed_time(end) * 1e3 / max(steps, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=151936)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--rows", type=int, default=32)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    ids, model, drawn, us = run(a.vocab, a.hidden, a.rows, a.steps)
    for r in range(min(a.rows, 3)):
        print("row %d: ids %s" % (r, ids[r].tolist()))
        print("       model logprobs %s" % [round(v, 3) for v in model[r].tolist()])
        print("       drawn logprobs %s" % [round(v, 3) for v in drawn[r].tolist()])
    print("%d rows, %d x %d table: %.1f us a decode step" % (a.rows, a.hidden, a.vocab, us))


if __name__ == "__main__":
    main()
