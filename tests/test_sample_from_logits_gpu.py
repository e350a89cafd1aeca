"""lmh_sample_from_logits against its definition (include/lmh.h), row by row on the host.

The definition's weights are whole numbers made from fp32 values 2^t.  The reference takes those
values from torch.exp2 (the same function of CUDA's math library), does everything after them in
Python and numpy integers and 64-bit floats, by sorting, and the drawn ids must be equal -- for
every split, type, alignment and filter.

Tolerance of the log-probability: |t ln 2| <= 23 for a token that can be drawn (its weight is at
least 1), with four fp32 roundings (5.5e-6), the logarithm (1e-6), and the sum of the kept weights,
each rounded by at most half a unit of 2^-32: V * 2^-33.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LOG2E = np.float32(1.4426950408889634)


def exp2_f32(t):
    return torch.exp2(torch.from_numpy(np.ascontiguousarray(t)).cuda()).cpu().numpy()


def reference_row(z, allowed, T, k, p, m, u):
    """(id, logprob) of one row; z fp32 numpy."""
    V = z.size
    z = z.copy()
    z[np.isnan(z)] = -np.inf
    if allowed is not None:
        z[~allowed] = -np.inf
    zm = z.max()
    if zm == -np.inf:
        return -1, math.nan
    if zm == np.inf:
        z = np.where(z == np.inf, np.float32(0), np.float32(-np.inf))
        zm = np.float32(0)
    if not T > 0:
        return int(np.flatnonzero(z == zm)[0]), 0.0
    with np.errstate(all="ignore"):
        c = np.float32(np.float32(1) / np.float32(T)) * LOG2E
        c = np.float32(min(max(c, np.float32(2.0 ** -126)), np.finfo(np.float32).max))
        t = ((z - zm).astype(np.float32) * c).astype(np.float32)
    w = np.rint(exp2_f32(t).astype(np.float64) * 2.0 ** 32).astype(np.int64)
    order = np.argsort(-z.astype(np.float64), kind="stable")
    cum = np.cumsum(w[order])
    keep = np.ones(V, dtype=bool)
    if 0 < k < V:
        keep[k:] = False
    if p < 1:
        mass = int(cum[keep.sum() - 1])
        need = max(1, math.ceil(float(np.float32(p)) * float(mass)))
        keep &= (cum - w[order]) < need
    if m > 0:
        lm = min(float(torch.log2(torch.tensor(m, dtype=torch.float32, device="cuda"))), 0.0)
        keep &= t[order] >= np.float32(lm)
    ids = np.sort(order[keep])
    cdf = np.cumsum(w[ids])
    total = int(cdf[-1])
    u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0 ** -24)
    r = min(int(math.floor(float(np.float32(u)) * float(total))), total - 1)
    j = int(ids[np.searchsorted(cdf, r, side="right")])
    return j, float(t[j]) * math.log(2.0) - math.log(total / 2.0 ** 32)


def pack_mask(allowed):
    rows, V = allowed.shape
    words = (V + 31) // 32
    bits = np.zeros((rows, words * 32), dtype=bool)
    bits[:, :V] = allowed
    out = np.zeros((rows, words), dtype=np.uint32)
    for b in range(32):
        out |= bits[:, b::32].astype(np.uint32) << np.uint32(b)
    return torch.from_numpy(out.view(np.int32)).cuda()


def check(lmh, logits, u, T=None, k=None, p=None, m=None, allowed=None, mask=None):
    """Draw on the GPU and compare every row."""
    rows, V = logits.shape
    dev = "cuda"

    def f32(x):
        return None if x is None else torch.tensor(x, dtype=torch.float32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if allowed is not None and mask is None:
        mask = pack_mask(allowed)
    o = lmh.sample_from_logits(logits, f32(u), temperature=f32(T),
                               top_k=None if k is None else torch.tensor(k, dtype=torch.int32, device=dev),
                               top_p=f32(p), min_p=f32(m), mask=mask, dev_status=status)
    ids, lps = o["sampled_ids"].cpu().numpy(), o["sampled_logprob"].cpu().numpy()
    z = logits.float().cpu().numpy()
    empty = False
    for i in range(rows):
        want, lp = reference_row(z[i], None if allowed is None else allowed[i], 1.0 if T is None else T[i],
                                 0 if k is None else k[i], 1.0 if p is None else p[i], 0.0 if m is None else m[i],
                                 u[i])
        what = (i, None if T is None else T[i], None if k is None else k[i], None if p is None else p[i],
                None if m is None else m[i], u[i])
        assert ids[i] == want, (what, int(ids[i]), want)
        if want < 0:
            empty = True
            assert math.isnan(lps[i])
        else:
            assert abs(lps[i] - lp) <= 6.5e-6 + V * 2.0 ** -33, (what, lps[i], lp)
    assert int(status.item()) == (0x20 if empty else 0)
    return ids


def settings(rng, rows, V):
    """Random per-row settings, off and extreme ones among them."""
    T = rng.choice([0.0, 0.3, 0.7, 1.0, 1.3, 5.0], rows).tolist()
    k = rng.choice([0, 0, 1, 2, 5, 20, 50, 100, 1024, 1025, 3000, V - 1, V, V + 5], rows).tolist()
    p = rng.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.8, 0.9, 0.95, 0.99, 0.999999], rows).tolist()
    m = rng.choice([0.0, 0.0, 0.0, 0.001, 0.05, 0.5, 1.0], rows).tolist()
    u = rng.random(rows, dtype=np.float32).tolist()
    return T, k, p, m, u


def model_logits(rng, rows, V):
    """A bulk and a few tokens that stand out, by more in some rows than in others."""
    z = rng.standard_normal((rows, V)).astype(np.float32) * 2
    for i in range(rows):
        n = min(V, 40)
        z[i, rng.integers(0, V, n)] += rng.uniform(0, 14) + rng.standard_normal(n).astype(np.float32)
    return z


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,V", [(3, 1), (5, 2), (9, 7), (16, 65), (16, 130), (33, 1000), (40, 4100), (24, 8193),
                                    (12, 32771)])
def test_small_vocabularies(lmh, rows, V, dtype):
    rng = np.random.default_rng(rows * 1000 + V)
    z = torch.from_numpy(model_logits(rng, rows, V)).to(DT[dtype]).cuda()
    T, k, p, m, u = settings(rng, rows, V)
    check(lmh, z, u, T, k, p, m)


@pytest.mark.parametrize("rows,V,dtype", [(1, 128256, "f32"), (32, 151936, "f32"), (20, 248320, "bf16"),
                                          (4, 393216, "f32"), (200, 50257, "f16"), (3, 393216, "bf16")])
def test_large_vocabularies(lmh, rows, V, dtype):
    rng = np.random.default_rng(rows + V)
    z = torch.from_numpy(model_logits(rng, rows, V)).to(DT[dtype]).cuda()
    T, k, p, m, u = settings(rng, rows, V)
    check(lmh, z, u, T, k, p, m)


@pytest.mark.parametrize("what", ["none", "top_k", "top_p", "min_p", "temperature"])
def test_one_filter_at_a_time(lmh, what):
    rng = np.random.default_rng(7)
    rows, V = 24, 20011
    z = torch.from_numpy(model_logits(rng, rows, V)).cuda()
    T, k, p, m, u = settings(rng, rows, V)
    check(lmh, z, u, T=T if what == "temperature" else None, k=k if what == "top_k" else None,
          p=p if what == "top_p" else None, m=m if what == "min_p" else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("levels", [1, 2, 5, 40])
def test_ties(lmh, levels, dtype):
    """Few distinct values: every threshold falls among equal logits, which are kept in id order."""
    rng = np.random.default_rng(levels)
    rows, V = 40, 9001
    z = torch.from_numpy(rng.integers(0, levels, (rows, V)).astype(np.float32) * 0.25).to(DT[dtype]).cuda()
    T, k, p, m, u = settings(rng, rows, V)
    check(lmh, z, u, T, k, p, m)


def test_flat_rows_keep_large_sets(lmh):
    """top-p over rows without a favourite: the kept set is most of the vocabulary."""
    rng = np.random.default_rng(11)
    rows, V = 16, 151936
    z = torch.from_numpy(rng.standard_normal((rows, V)).astype(np.float32) * 0.5).cuda()
    check(lmh, z, rng.random(rows, dtype=np.float32).tolist(), T=[1.0] * rows,
          p=[0.5, 0.8, 0.9, 0.95, 0.99, 0.999, 0.01, 0.3] * 2, k=[0] * 8 + [100000] * 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,V", [(24, 4100), (9, 70001)])
def test_mask(lmh, rows, V, dtype):
    """Grammar masks, from one allowed token to most of them; NaN and infinities at forbidden places, a row with
    nothing allowed, and spare mask words with bits set."""
    rng = np.random.default_rng(V)
    share = 10.0 ** -rng.uniform(0, 4, (rows, 1))
    allowed = rng.random((rows, V)) < share
    allowed[:, -1] |= ~allowed.any(1)
    allowed[2] = False
    allowed[3] = False
    allowed[3, V - 1] = True
    z = model_logits(rng, rows, V)
    bad = np.where(allowed, z, rng.choice([np.nan, np.inf, -np.inf, 0, 100], z.shape)).astype(np.float32)
    T, k, p, m, u = settings(rng, rows, V)
    mask = pack_mask(allowed)
    mask = torch.cat([mask, torch.full((rows, 3), -1, dtype=torch.int32, device="cuda")], 1)
    if V % 32:
        mask[:, V // 32] |= torch.tensor(-1 << (V % 32), dtype=torch.int32, device="cuda")
    ids = check(lmh, torch.from_numpy(bad).to(DT[dtype]).cuda(), u, T, k, p, m, allowed=allowed, mask=mask)
    assert ids[2] == -1 and ids[3] == V - 1


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_special_values(lmh, dtype):
    """NaN, infinities, the type's lowest value, denormals, empty rows, in places that are allowed."""
    rng = np.random.default_rng(5)
    V = 3001
    low = float(torch.finfo(DT[dtype]).min)
    rows = [np.full(V, -np.inf), np.full(V, np.nan), np.full(V, low), np.full(V, -low), np.full(V, np.inf)]
    r = rng.standard_normal(V)
    r[::3] = np.nan
    rows.append(r)
    r = rng.standard_normal(V)
    r[[5, 77, 2999]] = np.inf
    rows.append(r)
    r = np.full(V, low)
    r[1234] = 0.5
    rows.append(r)
    r = np.full(V, -np.inf)
    r[0] = low
    rows.append(r)
    r = rng.standard_normal(V) * 1e-39
    rows.append(r)
    r = np.where(rng.random(V) < 0.5, low, -low)
    rows.append(r)
    z = torch.from_numpy(np.stack(rows * 4).astype(np.float32)).to(DT[dtype]).cuda()
    n = z.shape[0]
    T, k, p, m, u = settings(rng, n, V)
    check(lmh, z, u, T=[1.0] * n)
    check(lmh, z, u, T, k, p, m)


@pytest.mark.parametrize("V", [2000, 60000])
def test_extreme_settings(lmh, V):
    rng = np.random.default_rng(3)
    nan, inf = math.nan, math.inf
    T = [-1.0, nan, 1e-45, 1e-38, 1e-30, 1e-3, 1e30, 3e38, inf, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0]
    n = len(T)
    k = [0] * 9 + [-5, 1, 0, 0, 0, 0, 0, 0, 0]
    p = [1.0] * 9 + [nan, 1.0, -1.0, 1e-20, 2.0, 1 - 2.0 ** -24, 0.9, 1.0, 1.0]
    m = [0.0] * 9 + [nan, 0.0, 0.0, 0.0, -1.0, 0.0, 1e-38, 2.0, inf]
    z = torch.from_numpy(model_logits(rng, n, V)).cuda()
    for u in ([0.0] * n, [1 - 2.0 ** -24] * n, [0.5] * n, [1.0] * n, [-3.0] * n, [nan] * n):
        check(lmh, z, u, T, k, p, m)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strides_and_alignment(lmh, dtype):
    """Rows that start at every phase of a 16-byte vector; the columns beside a row must not matter."""
    rng = np.random.default_rng(9)
    rows, V = 10, 5003
    for pad, first in [(0, 0), (1, 0), (3, 1), (5, 7), (8, 3)]:
        full = torch.full((rows, first + V + pad), 1e4, dtype=DT[dtype], device="cuda")
        view = full[:, first:first + V]
        view.copy_(torch.from_numpy(model_logits(rng, rows, V)))
        T, k, p, m, u = settings(rng, rows, V)
        check(lmh, view, u, T, k, p, m)


def test_a_draw_does_not_depend_on_the_batch(lmh):
    rng = np.random.default_rng(21)
    rows, V = 160, 40000
    z = torch.from_numpy(model_logits(rng, rows, V)).to(torch.bfloat16).cuda()
    T, k, p, m, u = [torch.tensor(x, device="cuda") for x in settings(rng, rows, V)]
    k, p, m, T = k.to(torch.int32), p.float(), m.float(), T.float()
    o = lmh.sample_from_logits(z, u, temperature=T, top_k=k, top_p=p, min_p=m)
    for i in (0, 17, 159):
        one = lmh.sample_from_logits(z[i:i + 1], u[i:i + 1], temperature=T[i:i + 1], top_k=k[i:i + 1],
                                     top_p=p[i:i + 1], min_p=m[i:i + 1])
        assert int(one["sampled_ids"]) == int(o["sampled_ids"][i])
        assert float(one["sampled_logprob"]) == float(o["sampled_logprob"][i])


def test_draws_follow_the_distribution(lmh):
    """Evenly spaced uniforms hit every kept token in proportion to its probability (to one draw in n)."""
    V, n = 500, 4096
    rng = np.random.default_rng(2)
    z = (rng.standard_normal(V) * 2).astype(np.float32)
    logits = torch.from_numpy(np.tile(z, (n, 1))).cuda()
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    o = lmh.sample_from_logits(logits, u, temperature=torch.full((n,), 0.8, device="cuda"))
    got = np.bincount(o["sampled_ids"].cpu().numpy(), minlength=V) / n
    e = np.exp((z.astype(np.float64) - z.max()) / 0.8)
    assert np.abs(got - e / e.sum()).max() <= 1.5 / n


def test_streams_graphs_and_no_rows(lmh):
    rng = np.random.default_rng(4)
    rows, V = 6, 30000
    z = torch.from_numpy(model_logits(rng, rows, V)).cuda()
    u = torch.rand(rows, device="cuda")
    p = torch.full((rows,), 0.9, device="cuda")
    want = lmh.sample_from_logits(z, u, top_p=p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = lmh.sample_from_logits(z, u, top_p=p, stream=side)
    side.synchronize()
    assert torch.equal(o["sampled_ids"], want["sampled_ids"])
    out = {"sampled_ids": torch.zeros(rows, dtype=torch.int32, device="cuda"), "sampled_logprob": None}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lmh.sample_from_logits(z, u, top_p=p, out=out)
    u.copy_(torch.rand(rows, device="cuda"))
    g.replay()
    assert torch.equal(out["sampled_ids"], lmh.sample_from_logits(z, u, top_p=p)["sampled_ids"])
    none = lmh.sample_from_logits(z[:0], u[:0])
    assert none["sampled_ids"].numel() == 0
