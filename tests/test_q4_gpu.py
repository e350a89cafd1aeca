"""4-bit tables: lmh_quantize_q4, lmh_project_q4 and lmh_lookup_q4 against 64-bit references.

The projection's inputs enter exactly (16-bit hidden rows, whole numbers q - zero); its fp32 sums
are within (H + 8) * 2^-23 of the sum of the terms' magnitudes (every addition rounded or cut off
once, the scale and logit_scale products among them), and the stored value is rounded once more in
a 16-bit out.  The lookup and the quantiser round at stated places only, so they are exact.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def random_table(lmh, V, H, group, zeros, scale="bf16", seed=0, pad=0):
    """(Q4Table, values in f64).  pad: spare columns, so that the rows of every array are strided."""
    rng = np.random.default_rng(seed)
    G = H // group
    packed = torch.from_numpy(rng.integers(0, 256, (V, H // 2 + 16 * pad), dtype=np.uint8)).cuda()[:, :H // 2]
    s = (rng.random((V, G + pad)) + 0.5).astype(np.float32) * 0.01 * rng.choice([-1, 1], (V, G + pad))
    scales = torch.from_numpy(s.astype(np.float32)).to(DT[scale]).cuda()[:, :G]
    z = None
    if zeros:
        z = torch.from_numpy(rng.integers(0, 16, (V, G + pad), dtype=np.uint8)).cuda()[:, :G]
    return lmh.Q4Table(packed, scales, z, group), values(packed, scales, z, group)


def values(packed, scales, zeros, group):
    p = packed.cpu().numpy()
    q = np.empty((p.shape[0], 2 * p.shape[1]))
    q[:, 0::2], q[:, 1::2] = p & 15, p >> 4
    z = 8.0 if zeros is None else np.repeat((zeros.cpu().numpy() & 15).astype(np.float64), group, 1)
    return (q - z) * np.repeat(scales.double().cpu().numpy(), group, 1)


def check_project(out, x, w, H, scale, dtype):
    want = scale * (x @ w.T)
    bound = abs(scale) * (np.abs(x) @ np.abs(w).T) * (H + 8) * 2.0 ** -23
    bound += (np.abs(want) + bound) * EPS[dtype] + 1e-45 + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 70])
@pytest.mark.parametrize("zeros", [False, True])
def test_project(lmh, rows, group, zeros):
    rng = np.random.default_rng(rows * group)
    V, H = 1003, group * int(rng.integers(1, 12))
    table, w = random_table(lmh, V, H, group, zeros, seed=rows)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = lmh.project_q4(x, table)
    assert out.dtype == torch.float32
    check_project(out, x.double().cpu().numpy(), w, H, 1.0, "f32")


@pytest.mark.parametrize("dtype,out,scale", [("bf16", "bf16", "bf16"), ("f16", "f16", "f16"), ("f16", "f32", "f32"),
                                             ("bf16", "f32", "f16"), ("f16", "f32", "bf16")])
@pytest.mark.parametrize("group,rows", [(32, 3), (64, 12), (128, 20)])
def test_project_types(lmh, group, rows, dtype, out, scale):
    rng = np.random.default_rng(rows)
    V, H = 517, 1024
    table, w = random_table(lmh, V, H, group, group == 64, scale=scale, seed=1)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(DT[dtype]).cuda()
    o = lmh.project_q4(x, table, out_dtype=DT[out], logit_scale=0.3)
    check_project(o, x.double().cpu().numpy(), w, H, float(np.float32(0.3)), out)


@pytest.mark.parametrize("V", [1, 15, 16, 17, 127, 128, 129, 4096, 30011])
@pytest.mark.parametrize("H,group", [(32, 32), (64, 64), (128, 128), (320, 64), (2560, 64), (4096, 128)])
def test_project_shapes(lmh, V, H, group):
    rng = np.random.default_rng(V + H)
    rows = int(rng.choice([1, 5, 8, 13, 32]))
    table, w = random_table(lmh, V, H, group, bool(V % 2), seed=H)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    check_project(lmh.project_q4(x, table), x.double().cpu().numpy(), w, H, 1.0, "f32")


@pytest.mark.parametrize("rows,H,group", [(1, 16384, 128), (9, 8192, 64), (32, 8192, 32), (20, 13824, 128),
                                          (4, 14336, 32)])
def test_project_long_rows(lmh, rows, H, group):
    """Hidden rows that do not fit in shared memory at once."""
    rng = np.random.default_rng(H)
    table, w = random_table(lmh, 700, H, group, True, seed=H)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    check_project(lmh.project_q4(x, table), x.double().cpu().numpy(), w, H, 1.0, "f32")


@pytest.mark.parametrize("rows,V,H,group", [(1, 151936, 256, 32), (8, 120001, 1024, 32), (12, 90000, 512, 64),
                                            (16, 100003, 1280, 128), (32, 60001, 768, 64), (3, 200003, 64, 32),
                                            (20, 151936, 128, 64)])
def test_project_many_tiles_per_sm(lmh, rows, V, H, group):
    """Vocabularies that give every SM several tiles; repeated calls, the same bits each time."""
    rng = np.random.default_rng(V)
    table, w = random_table(lmh, V, H, group, group == 128, seed=rows)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = lmh.project_q4(x, table, dev_status=status)
    check_project(first, x.double().cpu().numpy(), w, H, 1.0, "f32")
    for _ in range(20):
        assert torch.equal(lmh.project_q4(x, table, dev_status=status), first)
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_project_hidden_ranges(lmh, dtype):
    """Rows of very large, very small, subnormal and widely spread values, and zeros."""
    rng = np.random.default_rng(31)
    V, H = 400, 640
    table, w = random_table(lmh, V, H, 64, True, scale="f32", seed=9)
    big, small = (1e30, 1e-36) if dtype == "bf16" else (3e4, 1e-7)
    x = rng.standard_normal((12, H))
    for i, f in enumerate([big, small, 1e-40 if dtype == "bf16" else 6e-8, 0.0]):
        x[i] = np.clip(x[i] * f, -6e4 if dtype == "f16" else -3e38, 6e4 if dtype == "f16" else 3e38)
    x[4] *= 10.0 ** rng.uniform(-20 if dtype == "bf16" else -4, 4, H)
    x[5, ::2] = 0
    x[6] = 0
    x[6, 17] = 1.5
    xt = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    check_project(lmh.project_q4(xt, table), xt.double().cpu().numpy(), w, H, 1.0, "f32")


def test_project_strides_and_row_index(lmh):
    """Strided hidden rows (odd strides too), strided table rows and output rows, gathered rows; an index out of range
    reads zeros and sets the status bit; nothing is written beside the output's columns."""
    rng = np.random.default_rng(8)
    V, H, T = 777, 256, 50
    table, w = random_table(lmh, V, H, 64, True, seed=3, pad=1)
    for pad, first in [(0, 0), (3, 1), (8, 8)]:
        full = torch.from_numpy(rng.standard_normal((T, first + H + pad)).astype(np.float32)).to(torch.bfloat16).cuda()
        hidden = full[:, first:first + H]
        for n in (4, 21):
            idx = rng.integers(0, T, n).astype(np.int32)
            idx[1], idx[3] = -1, T
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            buf = torch.full((n, V + 5), 7.0, device="cuda")
            lmh.project_q4(hidden, table, row_idx=torch.from_numpy(idx).cuda(), out=buf[:, 2:2 + V], dev_status=status)
            x = hidden.double().cpu().numpy()[np.clip(idx, 0, T - 1)]
            x[[1, 3]] = 0
            check_project(buf[:, 2:2 + V], x, w, H, 1.0, "f32")
            assert (buf[:, :2] == 7).all() and (buf[:, 2 + V:] == 7).all()
            assert int(status.item()) == 0x8


def test_project_bad_hidden_values_stay_in_their_row(lmh):
    V, H = 300, 512
    table, w = random_table(lmh, V, H, 64, False, seed=5)
    x = torch.randn(11, H, device="cuda").to(torch.bfloat16)
    x[2, 100] = math.nan
    x[5, 3] = math.inf
    x[10] = torch.finfo(torch.bfloat16).min
    out = lmh.project_q4(x, table)
    assert torch.isnan(out[2]).all()
    good = [i for i in range(11) if i not in (2, 5, 10)]
    check_project(out[good], x[good].double().cpu().numpy(), w, H, 1.0, "f32")


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,group,zeros,scale", [(32, 32, False, "bf16"), (320, 64, True, "f16"),
                                                 (1024, 128, True, "f32"), (2560, 64, False, "bf16")])
def test_lookup(lmh, H, group, zeros, scale, out):
    """Exact in every bit: (q - zero) * scale and the multiplier rounded to fp32, then to the output's type."""
    V = 1111
    table, _ = random_table(lmh, V, H, group, zeros, scale=scale, seed=H, pad=1)
    rng = np.random.default_rng(H)
    for n in (1, 2, 33, 700):
        ids = rng.integers(0, V, n).astype(np.int32)
        if n > 2:
            ids[1] = -1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mult = math.sqrt(H)
        buf = torch.full((n, H + 3), 5.0, dtype=DT[out], device="cuda")
        for o in (lmh.lookup_q4(torch.from_numpy(ids).cuda(), table, scale=mult, out_dtype=DT[out], dev_status=status),
                  lmh.lookup_q4(torch.from_numpy(ids).cuda(), table, scale=mult, out=buf[:, 1:1 + H],
                                dev_status=status)):
            p = table.packed[torch.from_numpy(np.maximum(ids, 0)).long().cuda()].cpu()
            q = torch.stack((p & 15, p >> 4), -1).view(n, -1).float()
            at = torch.from_numpy(np.maximum(ids, 0)).long().cuda()
            z = 8.0 if not zeros else (table.zeros[at].cpu().float()).repeat_interleave(group, 1)
            w = (q - z) * table.scales[at].float().cpu().repeat_interleave(group, 1) * mult
            w[ids == -1] = 0
            assert torch.equal(o.cpu(), w.to(DT[out]))
        assert (buf[:, 0] == 5).all() and (buf[:, 1 + H:] == 5).all()
        assert int(status.item()) == 0
    status.zero_()
    o = lmh.lookup_q4(torch.tensor([V, -2, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), table, dev_status=status)
    assert int(status.item()) == 0x2 and (o == 0).all()


def reference_quantise(W, group, zeros, dtype):
    w = W.float().view(W.shape[0], -1, group)
    hi, lo = w.amax(-1).clamp(min=0), w.amin(-1).clamp(max=0)
    s = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7).to(dtype)
    sf = s.float()
    ok = sf > 0
    safe = torch.where(ok, sf, torch.ones_like(sf))
    zero = torch.where(ok, torch.round(-lo / safe).clamp(0, 15), torch.zeros_like(sf)) if zeros else \
        torch.full_like(sf, 8)
    r = torch.where(ok[..., None], torch.round(w / safe[..., None]), torch.zeros_like(w))
    return (r + zero[..., None]).clamp(0, 15).view(W.shape).to(torch.uint8), s, zero.to(torch.uint8)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,H,group", [(1, 32, 32), (77, 192, 64), (130, 1024, 128), (1000, 2560, 64)])
def test_quantise(lmh, V, H, group, scale, zeros):
    for first, pad in [(0, 0), (3, 2)]:
        full = (torch.randn(V, first + H + pad, device="cuda") * 0.02).to(torch.bfloat16)
        W = full[:, first:first + H]
        W[0, :group] = 0
        W[-1, -group:] = W[-1, -group:].abs()
        W[V // 2] = -W[V // 2].abs()
        t = lmh.quantize_q4(W, group=group, zeros=zeros, scale_dtype=DT[scale])
        q, s, z = reference_quantise(W.cpu(), group, zeros, DT[scale])  # IEEE division on either side
        got = torch.stack((t.packed & 15, t.packed >> 4), -1).view(V, H).cpu()
        assert torch.equal(t.scales.cpu(), s)
        if zeros:
            assert torch.equal(t.zeros.cpu(), z)
        assert torch.equal(got, q)


def test_quantise_then_project_is_close_to_the_table(lmh):
    """Half a step of each group's scale is the most an entry moves (its scale's rounding apart)."""
    W = (torch.randn(500, 512, device="cuda") * 0.02).to(torch.bfloat16)
    t = lmh.quantize_q4(W, group=32, scale_dtype=torch.float32)
    w = values(t.packed, t.scales, None, 32)
    step = np.repeat(t.scales.double().cpu().numpy(), 32, 1)
    assert (np.abs(w - W.double().cpu().numpy()) <= 0.5001 * step).all()


def test_decode_loop(lmh):
    """lookup -> (a body) -> project -> sample on the device, several steps in one captured graph."""
    V, H, n = 5000, 256, 6
    table = lmh.quantize_q4((torch.randn(V, H, device="cuda") * 0.05).to(torch.bfloat16), group=64)
    u = torch.rand(4, n, device="cuda")
    T = torch.full((n,), 0.9, device="cuda")
    p = torch.full((n,), 0.95, device="cuda")

    def steps(ids):
        out = []
        for i in range(4):
            x = lmh.lookup_q4(ids, table, scale=16.0)
            o = lmh.sample_from_logits(lmh.project_q4(x, table), u[i], temperature=T, top_p=p)
            ids = o["sampled_ids"]
            out.append(ids)
        return out
    first = torch.arange(n, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in steps(first)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(first)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H,group", [(32, 32), (96, 32), (320, 64), (128, 128)])
@pytest.mark.parametrize("scale", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [1, 12, 20])
def test_project_infinite_scale_of_the_last_group(lmh, rows, scale, H, group):
    """The entries that fill a row's last 256 up count for nothing, whatever the last scale is."""
    V, G = 200, H // group
    packed = torch.full((V, H // 2), 0xFF, dtype=torch.uint8, device="cuda")  # every entry 15 - 8 = 7
    scales = torch.ones(V, G, dtype=DT[scale], device="cuda")
    scales[5, -1], scales[130, -1] = float("inf"), float("-inf")
    x = torch.ones(rows, H, dtype=torch.bfloat16, device="cuda")
    want = torch.full((rows, V), 7.0 * H, device="cuda")
    want[:, 5], want[:, 130] = float("inf"), float("-inf")
    assert torch.equal(lmh.project_q4(x, lmh.Q4Table(packed, scales, None, group)), want)  # whole numbers: exact


def test_project_reads_the_table_made_just_before(lmh):
    """No synchronisation between making a table and projecting through it."""
    V, H = 20011, 1024
    ws = [torch.randn(V, H, generator=torch.Generator("cuda").manual_seed(i), device="cuda").to(torch.bfloat16)
          for i in range(2)]
    x = torch.randn(8, H, device="cuda").to(torch.bfloat16)
    want = []
    for w in ws:
        t = lmh.quantize_q4(w, 64)
        torch.cuda.synchronize()
        want.append(lmh.project_q4(x, t))
    del t  # (its memory holds the next tables: the allocator gives it out again)
    got = []
    for i in range(8):
        t = lmh.quantize_q4(ws[i & 1], 64)
        got.append(lmh.project_q4(x, t))
        del t
    for i in range(8):
        assert torch.equal(got[i], want[i & 1]), i


def test_project_very_long_rows(lmh):
    """The hidden rows in many pieces; no limit on H."""
    rng = np.random.default_rng(4)
    H = 81920 + 96
    table, w = random_table(lmh, 130, H, 32, True, seed=4)
    x = torch.from_numpy(rng.standard_normal((9, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    check_project(lmh.project_q4(x, table), x.double().cpu().numpy(), w, H, 1.0, "f32")


@pytest.mark.parametrize("rows,V,H,group", [(32, 60000, 896, 64), (20, 151936, 128, 32), (17, 50003, 384, 128),
                                            (24, 40000, 2816, 64), (24, 2000, 2848, 32), (32, 90000, 32, 32),
                                            (25, 70001, 1120, 32), (64, 30000, 640, 128), (41, 25000, 192, 64)])
@pytest.mark.parametrize("zeros", [False, True])
def test_project_wide_many_tiles(lmh, rows, V, H, group, zeros):
    """More than 16 rows: odd numbers of 128 entries, long and short rings, several tiles per SM, and
    hidden rows that just fit and just do not."""
    rng = np.random.default_rng(H)
    table, w = random_table(lmh, V, H, group, zeros, seed=H)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = lmh.project_q4(x, table)
    check_project(out, x.double().cpu().numpy(), w, H, 1.0, "f32")
    for _ in range(3):
        assert torch.equal(lmh.project_q4(x, table), out)
