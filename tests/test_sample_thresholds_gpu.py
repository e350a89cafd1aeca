"""lmh_sample_from_logits where the search for a threshold goes its long ways.

Flat rows (high temperatures) put more unequal logits into one part of the scale than a list holds, so
the search goes on level by level; logits far from 0 fall into the ends of the lists' bins.  The
reference and its tolerance are those of test_sample_from_logits_gpu.py.
"""
import numpy as np
import pytest
import torch

from test_sample_from_logits_gpu import DT, check, model_logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,V", [(18, 9001), (160, 9001), (18, 60000), (18, 150001)])
@pytest.mark.parametrize("both", [False, True])
def test_high_temperatures(lmh, rows, V, dtype, both):
    """Top-k beyond a list, top-p, and the one after the other, on rows that a temperature of 1e3 to 1e30 flattens;
    from one CTA a row to several, above and below the size from which a sample is taken."""
    rng = np.random.default_rng(V + rows)
    z = torch.from_numpy(model_logits(rng, rows, V)).to(DT[dtype]).cuda()
    T = np.resize([1e3, 1e6, 1e30, 30.0], rows).tolist()
    k = np.resize([500, 0, 1024, 0, min(20000, V - 7), 0], rows).tolist()
    p = np.resize([1.0, 0.3, 1.0, 0.9, 1.0, 0.999], rows).tolist()
    if both:
        k = np.resize([500, 1024, min(20000, V - 7)], rows).tolist()
        p = np.resize([0.3, 0.9, 0.5, 0.9, 0.3], rows).tolist()
    for u in (rng.random(rows, dtype=np.float32).tolist(), [1 - 2.0 ** -24] * rows):
        check(lmh, z, u, T, k, p)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [-1000.0, -100.0, -64.0, 64.0, 100.0, 1000.0])
@pytest.mark.parametrize("V", [9001, 60000])
def test_logits_far_from_zero(lmh, shift, V, dtype):
    rng = np.random.default_rng(V)
    rows = 24
    z = torch.from_numpy(model_logits(rng, rows, V) + np.float32(shift)).to(DT[dtype]).cuda()
    k = rng.choice([0, 0, 1, 5, 50, 300, 384, 385, 1000], rows).tolist()
    p = rng.choice([1.0, 0.5, 0.8, 0.95, 0.99], rows).tolist()
    m = rng.choice([0.0, 0.0, 0.05], rows).tolist()
    check(lmh, z, rng.random(rows, dtype=np.float32).tolist(), [0.8] * rows, k, p, m)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("spread", [0.2, 0.01, 1e-6])
def test_narrow_rows(lmh, spread, dtype):
    """All of a row's logits within a bin or two of the lists."""
    rng = np.random.default_rng(3)
    rows, V = 16, 40000
    z = torch.from_numpy((1 + spread * rng.standard_normal((rows, V))).astype(np.float32)).to(DT[dtype]).cuda()
    k = np.resize([0, 50, 1000, 0], rows).tolist()
    p = np.resize([0.9, 1.0, 0.7, 0.1, 1.0], rows).tolist()
    check(lmh, z, rng.random(rows, dtype=np.float32).tolist(), [1.0] * rows, k, p)


def _time_us(call, calls=10, repeats=7):
    """The least of several times per call, of calls in a row (the host is ahead of the GPU)."""
    best = float("inf")
    for _ in range(repeats):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda._sleep(2000000)
        begin.record()
        for _ in range(calls):
            call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, begin.elapsed_time(end) * 1e3 / calls)
    return best


@pytest.mark.parametrize("rows,dtype", [(1, "f32"), (256, "bf16")])
def test_top_p_after_top_k_searches_once(lmh, rows, dtype):
    """Top-k and top-p each search a threshold: both together take less than twice the first alone.  (1.8 times.  With a
    sample of other tokens than those that top-k left, the second search was always made twice: 2.4 times.)"""
    V = 151936
    gen = torch.Generator("cuda").manual_seed(2)
    z = (torch.randn(rows, V, generator=gen, device="cuda") * 0.5).to(DT[dtype])
    u = torch.rand(rows, generator=gen, device="cuda")
    p = torch.full((rows,), 0.9, device="cuda")
    k = torch.full((rows,), 1000, dtype=torch.int32, device="cuda")
    one = _time_us(lambda: lmh.sample_from_logits(z, u, top_k=k))
    both = _time_us(lambda: lmh.sample_from_logits(z, u, top_k=k, top_p=p))
    assert both < 2.05 * one, (one, both)
