"""Calls that follow one another at once: what a call reads of the results of the one before it.

A kernel may start while the one before it ends, so a call that reads its inputs ahead of the wait
for that kernel would read what an earlier step left.  The steps run in a captured graph (its kernels
follow one another at once), with new hidden rows before every replay, and are compared with the same
calls one by one, the device idle in between.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

STEPS = 8


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def _replays_equal_single_calls(steps, inputs):
    """steps(sync) -> tensors, from `inputs`; the graph's results against those of single calls."""
    def refill(seed):
        for i, x in enumerate(inputs):
            x.copy_(_randn(1000 * seed + i, *x.shape))
    refill(0)
    steps(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(lambda: None)
    for replay in range(1, 5):
        refill(replay)
        want = [t.clone() for t in steps(torch.cuda.synchronize)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), "replay %d, result %d" % (replay, i)


def _ids(lmh, producer, x, W, seed):
    """Token ids (int32 [rows]) as the last thing that the call writes."""
    if producer == "sampled":
        return lmh.project_logprobs(x, W, sampling={"seed": seed}, k_max=20)["sampled_ids"]
    if producer == "best":
        return lmh.project_logprobs(x, W, k_max=1)["topk_ids"].view(-1)
    if producer == "given_logits":  # the best of logits that are in memory
        return lmh.logprobs_from_logits(x, k_max=1)["topk_ids"].view(-1)
    table, u = W
    return lmh.sample_from_logits(lmh.project_q4(x, table), u)["sampled_ids"]


def _producer(lmh, producer, rows, V, H):
    """(the steps' inputs, what else the producer takes)"""
    if producer == "given_logits":
        return [_randn(i, rows, V).to(torch.bfloat16) for i in range(STEPS)], None
    xs = [_randn(i, rows, H).to(torch.bfloat16) for i in range(STEPS)]
    W = _randn(77, V, H).to(torch.bfloat16)
    if producer == "draw":
        return xs, (lmh.quantize_q4(W, 64), torch.rand(rows, generator=torch.Generator("cuda").manual_seed(5),
                                                       device="cuda"))
    return xs, W


PRODUCERS = [("sampled", 32, 50000, 256), ("sampled", 4, 151936, 128), ("sampled", 100, 256, 256),
             ("best", 64, 20000, 512), ("best", 300, 256, 128), ("given_logits", 16, 40000, 0),
             ("given_logits", 1, 8000, 0), ("draw", 8, 30000, 256)]


@pytest.mark.parametrize("producer,rows,V,H", PRODUCERS)
def test_selected_ids_of_the_logits_reduction(lmh, producer, rows, V, H):
    xs, W = _producer(lmh, producer, rows, V, H)
    z = _randn(9, rows, V)

    def steps(sync):
        out = []
        for i, x in enumerate(xs):
            ids = _ids(lmh, producer, x, W, i)
            sync()
            out += [ids, lmh.logprobs_from_logits(z, sel=ids)["sel_logprob"]]
            sync()
        return out
    _replays_equal_single_calls(steps, xs)


@pytest.mark.parametrize("producer,rows,V,H", PRODUCERS)
def test_selected_ids_of_the_projection(lmh, producer, rows, V, H):
    xs, W = _producer(lmh, producer, rows, V, H)
    y, head = _randn(9, rows, 256).to(torch.bfloat16), _randn(10, V, 256).to(torch.bfloat16)

    def steps(sync):
        out = []
        for i, x in enumerate(xs):
            ids = _ids(lmh, producer, x, W, i)
            sync()
            out += [ids, lmh.project_logprobs(y, head, sel=ids)["sel_logprob"]]
            sync()
        return out
    _replays_equal_single_calls(steps, xs)


@pytest.mark.parametrize("rows,V,H", [(128, 256, 4096), (16, 256, 8192), (5, 40, 2048), (64, 20000, 512)])
def test_logits_that_the_projection_writes(lmh, rows, V, H):
    """The head's own logits (from one vocabulary range and from several), reduced and drawn from."""
    xs = [_randn(i, rows, H).to(torch.bfloat16) for i in range(STEPS)]
    W = (_randn(77, V, H) * H ** -0.5).to(torch.bfloat16)
    u = torch.rand(rows, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    z = torch.empty(rows, V, device="cuda")

    def steps(sync):
        out = []
        for x in xs:
            lmh.project_logprobs(x, W, logits_out=z)
            sync()
            out.append(lmh.logprobs_from_logits(z)["lse"])
            sync()
            lmh.project_logprobs(x, W, logits_out=z)
            sync()
            out.append(lmh.sample_from_logits(z, u)["sampled_ids"])
            sync()
        return out
    _replays_equal_single_calls(steps, xs)
