"""Adapters beside a projection (lmh_add_adapters) against the formula in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _case(rows, H, N, R, L, dtype=BF16, y_dtype=F32, seed=0, tokens=None, scales=True, ranks=False, none=True):
    g = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    c = {"x": randn(tokens or rows, H).to(dtype), "down": (randn(L, R, H) * H ** -0.5).to(dtype),
         "up": (randn(L, N, R) * 0.1).to(dtype), "y": (2 * randn(rows, N)).to(y_dtype), "row_idx": None,
         "idx": torch.randint(-1 if none else 0, L, (rows,), generator=g, device="cuda", dtype=torch.int32),
         "scales": 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda") if scales else None, "ranks": None}
    if ranks:
        c["ranks"] = torch.randint(0, R + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
    if tokens:
        c["row_idx"] = torch.randint(0, tokens, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return c


def _formula(c):
    """(out in 64 bits before its rounding, how far it may be off).

    Every fp32 sum of n terms is within n 2^-23 of its terms' magnitudes (twice fp32's half step, for sums
    that are cut and not rounded).  d is rounded to its type, half a step being 2^-8 of it for bf16 and 2^-11
    for f16; for fp32 outputs what that left is too, so that 2^-16 and 2^-22 remain (2^-38 of the row's largest
    for the smallest f16 parts).  Its product
    with the scale is within 2^-24, and y is added with one rounding."""
    step = {BF16: 2.0 ** -8, F16: 2.0 ** -11}[c["x"].dtype]
    if c["y"].dtype == F32:
        step *= step
    y, x = c["y"].double(), c["x"].double()
    idx, L = c["idx"].long(), c["down"].shape[0]
    out, off = y.clone(), torch.zeros_like(y)
    R, H = c["down"].shape[1:]
    for l in range(L):
        rows = (idx == l).nonzero().flatten()
        if not len(rows):
            continue
        r = R if c["ranks"] is None else max(0, min(R, int(c["ranks"][l])))
        s = 1.0 if c["scales"] is None else float(c["scales"][l])
        xr = x[rows if c["row_idx"] is None else c["row_idx"].long()[rows]]
        down, up = c["down"][l, :r].double(), c["up"][l, :, :r].double()
        d = xr @ down.t()
        e = xr.abs() @ down.abs().t() * (H + 8) * 2.0 ** -23 + d.abs() * (step + 2.0 ** -23)
        if c["x"].dtype == F16 and r:
            e += d.abs().amax(1, keepdim=True) * 2.0 ** -38  # (f16's smallest step is 2^-24, of 2^14)
        out[rows] += s * d @ up.t()
        off[rows] = s * (e @ up.abs().t() + d.abs() @ up.abs().t() * (2 * R + 8) * 2.0 ** -23)
    return out, off


def _check(c, got, what=""):
    want, off = _formula(c)
    half = torch.finfo(got.dtype).eps / 2
    off = off + (want.abs() + off) * (2.0 ** -24 + half) + (2.0 ** -25 if got.dtype == F16 else 0)
    bad = ~((got.double() - want).abs() <= off)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(),
                           float((got.double() - want).abs().max()), float(off.max()))
    none = c["idx"] == -1
    assert torch.equal(got[none], c["y"][none])


def _run(lmh, c, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = lmh.AdapterTable(c["down"], c["up"], scales=c["scales"], ranks=c["ranks"])
    out = lmh.add_adapters(c["x"], t, c["idx"], c["y"], row_idx=c["row_idx"], dev_status=st, **kw)
    assert int(st.item()) == 0
    return out


@pytest.mark.parametrize("dtype,y_dtype", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("rows,H,N,R,L", [
    (300, 64, 520, 8, 70), (513, 128, 1001, 16, 3), (400, 72, 264, 32, 2), (290, 256, 777, 64, 5), (257, 128, 512, 128, 4),
    (1, 8, 1, 8, 1), (1, 2560, 2560, 16, 4), (5, 128, 4096, 8, 3), (7, 1000, 33, 24, 2), (33, 512, 5003, 16, 8),
    (64, 4096, 1001, 32, 48), (70, 264, 640, 64, 1), (100, 1024, 515, 128, 3), (257, 136, 300, 40, 100)])
def test_against_the_formula(lmh, rows, H, N, R, L, dtype, y_dtype):
    c = _case(rows, H, N, R, L, dtype, y_dtype, seed=rows)
    _check(c, _run(lmh, c))


@pytest.mark.parametrize("rows,H,N,R,L", [(9, 256, 700, 16, 4), (40, 512, 333, 64, 12), (200, 128, 96, 128, 6),
                                          (333, 96, 400, 64, 9), (600, 64, 260, 16, 5), (260, 64, 264, 128, 5)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_ranks_and_what_stands_behind_them(lmh, rows, H, N, R, L, dtype):
    c = _case(rows, H, N, R, L, dtype, seed=3, ranks=True, tokens=2 * rows)
    c["ranks"][0] = 0
    c["ranks"][1] = 1
    c["ranks"][2] = 2 * R  # held to the rank
    for l, r in enumerate(c["ranks"].tolist()):
        c["down"][l, r:] = float("nan")
        c["up"][l, :, r:] = float("inf")
    _check(c, _run(lmh, c))


@pytest.mark.parametrize("rows", [1, 8, 9, 31, 32, 33, 64, 65, 256, 257, 500, 17000])
def test_one_adapter_many_rows(lmh, rows):
    c = _case(rows, 320, 770, 16, 2, seed=rows, none=False)
    c["idx"].fill_(1)
    c["down"][0] = float("nan")  # not in use
    _check(c, _run(lmh, c))


@pytest.mark.parametrize("rows", [50, 700])
def test_no_row_has_an_adapter(lmh, rows):
    c = _case(rows, 128, 100, 8, 2)
    c["idx"].fill_(-1)
    assert torch.equal(_run(lmh, c), c["y"])
    y = c["y"].clone()
    _run(lmh, dict(c, y=y), out=y)
    assert torch.equal(y, c["y"])


def test_long_packed_prompts(lmh):
    c = _case(3000, 512, 1024, 64, 5, BF16, BF16, seed=8)
    c["idx"] = c["idx"].sort().values
    _check(c, _run(lmh, c))


def test_whole_numbers_are_exact(lmh):
    """Products and sums of small whole numbers round nowhere."""
    g = torch.Generator("cuda").manual_seed(1)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")
    for dtype, R in ((BF16, 16), (F16, 16), (BF16, 64), (F16, 128)):
        c = {"x": whole(-2, 2, 37, 256).to(dtype), "down": whole(-2, 2, 6, R, 256).to(dtype),
             "up": whole(-4, 4, 6, 515, R).to(dtype), "y": whole(-9, 9, 37, 515).float(), "row_idx": None,
             "idx": whole(-1, 5, 37).int(), "scales": 2.0 ** whole(-1, 1, 6).float(), "ranks": None}
        assert torch.equal(_run(lmh, c).double(), _formula(c)[0])


@pytest.mark.parametrize("rows", [21, 290])
def test_strides_alignment_and_in_place(lmh, rows):
    c = _case(rows, 264, 99, 24, 5, seed=4)
    big_x = torch.zeros(rows, 271, dtype=BF16, device="cuda")
    big_x[:, 3:267] = c["x"]
    big_y = torch.zeros(rows, 103, device="cuda")
    big_y[:, 2:101] = c["y"]
    down = torch.zeros(5, 30, 280, dtype=BF16, device="cuda")[:, 2:26, 8:272]
    up = torch.zeros(7, 99, 40, dtype=BF16, device="cuda")[1:6, :, 8:32]
    down.copy_(c["down"]), up.copy_(c["up"])
    want = _run(lmh, c)
    s = dict(c, x=big_x[:, 3:267], down=down, up=up, y=big_y[:, 2:101])
    assert torch.equal(_run(lmh, s), want)
    out = torch.full((rows, 110), 7.0, device="cuda")
    assert torch.equal(_run(lmh, s, out=out[:, 5:104]), want)
    assert (out[:, :5] == 7).all() and (out[:, 104:] == 7).all()
    assert _run(lmh, s, out=s["y"]) is s["y"]
    assert torch.equal(big_y[:, 2:101], want) and (big_y[:, :2] == 0).all() and (big_y[:, 101:] == 0).all()


def test_shared_weights_and_one_row_strides(lmh):
    """All adapters may be one (a stride of zero), and dimensions of one entry may have any stride."""
    c = _case(12, 64, 50, 8, 1, none=False)
    t = lmh.AdapterTable(c["down"].expand(4, 8, 64), c["up"].expand(4, 50, 8))
    idx = torch.arange(12, device="cuda", dtype=torch.int32) % 4
    got = lmh.add_adapters(c["x"], t, idx, c["y"])
    assert torch.equal(got, _run(lmh, dict(c, scales=None)))


def test_bad_indices(lmh):
    from top_reduction_gb300 import lmh as L
    c = _case(9, 128, 200, 16, 3, none=False, tokens=20)
    t = lmh.AdapterTable(c["down"], c["up"], scales=c["scales"])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = c["idx"].clone()
    idx[2], idx[5] = 3, -7
    got = lmh.add_adapters(c["x"], t, idx, c["y"], row_idx=c["row_idx"], dev_status=st)
    assert int(st.item()) == L.DS_ADAPTER_OUT_OF_RANGE
    idx[2], idx[5] = -1, -1
    _check(dict(c, idx=idx), got)
    st.zero_()
    ri = c["row_idx"].clone()
    ri[0], ri[8] = 20, -1
    got = lmh.add_adapters(c["x"], t, c["idx"], c["y"], row_idx=ri, dev_status=st)
    assert int(st.item()) == L.DS_ROW_IDX_OUT_OF_RANGE
    assert torch.equal(got[[0, 8]], c["y"][[0, 8]])
    ok = [i for i in range(9) if i not in (0, 8)]
    assert torch.equal(got[ok], _run(lmh, c)[ok])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_large_small_and_infinite_values(lmh, dtype):
    """d beyond f16's range, tiny d, and rows with an infinity or NaN, which leave the other rows alone."""
    c = _case(12, 256, 128, 16, 2, dtype, seed=2, none=False)
    c["x"][0] *= 3000
    c["down"] *= 8
    c["x"][1] *= 1e-3
    plain = _run(lmh, c)
    _check(c, plain)
    c["x"][2, 5] = float("inf")
    c["x"][3, 7] = float("nan")
    got = _run(lmh, c)
    assert not torch.isfinite(got[2]).any() and torch.isnan(got[3]).all()
    others = [i for i in range(12) if i not in (2, 3)]
    assert torch.equal(got[others], plain[others])


@pytest.mark.parametrize("rows", [80, 400])
def test_a_rows_result_does_not_depend_on_its_place(lmh, rows):
    c = _case(rows, 512, 300, 32, 7, seed=6)
    whole = _run(lmh, c)
    perm = torch.randperm(rows, generator=torch.Generator().manual_seed(0)).cuda()
    again = _run(lmh, dict(c, x=c["x"][perm], idx=c["idx"][perm], y=c["y"][perm]))
    assert torch.equal(again, whole[perm])


def test_streams_workspace_and_graph(lmh):
    c, e = _case(30, 256, 500, 16, 4, seed=1), _case(11, 256, 500, 16, 4, seed=2)
    want = [_run(lmh, c), _run(lmh, e)]
    t = [lmh.AdapterTable(k["down"], k["up"], scales=k["scales"]) for k in (c, e)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lmh.add_adapters(c["x"], t[0], c["idx"], c["y"], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    ws = torch.empty(max(t[0].workspace_bytes(30), t[1].workspace_bytes(11)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # calls that follow one another at once share one workspace
        outs = [lmh.add_adapters(k["x"], a, k["idx"], k["y"], workspace=ws)
                for k, a in ((c, t[0]), (e, t[1]), (c, t[0]), (e, t[1]))]
    for _ in range(3):
        for o in outs:
            o.zero_()
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, want[i % 2])


@pytest.mark.parametrize("change,what", [
    (dict(x=torch.zeros(4, 8)), "one device"), (dict(x="wide"), "must be bfloat16"), (dict(x="half"), "must be bfloat16"),
    (dict(row_idx="long"), "row_idx must be"), (dict(out="other"), "out must be like y"),
    (dict(adapter_idx="short"), "4 entries"), (dict(workspace="small"), "workspace must be"), (dict(y="cols"), "contiguous")])
def test_binding_refusals(lmh, change, what):
    c = _case(4, 64, 40, 8, 2)
    t = lmh.AdapterTable(c["down"], c["up"])
    a = dict(x=c["x"], table=t, adapter_idx=c["idx"], y=c["y"])
    made = {"wide": lambda: torch.zeros(4, 72, dtype=BF16, device="cuda"), "half": lambda: c["x"].half(),
            "long": lambda: torch.zeros(4, dtype=torch.int64, device="cuda"), "other": lambda: c["y"].bfloat16(),
            "short": lambda: c["idx"][:3], "small": lambda: torch.empty(16, dtype=torch.uint8, device="cuda"),
            "cols": lambda: torch.zeros(40, 4, device="cuda").t()}
    for k, v in change.items():
        if isinstance(v, torch.Tensor):
            with pytest.raises((ValueError, TypeError, AttributeError)):
                lmh.add_adapters(**dict(a, x=v))
            return
        a[k] = made[v]()
    with pytest.raises(ValueError, match=what):
        lmh.add_adapters(**a)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,H,N,R,L", [(300, 64, 4, 8, 3), (257, 128, 516, 16, 4), (700, 72, 1004, 32, 2),
                                          (290, 256, 780, 64, 5), (513, 96, 260, 128, 3)])
def test_16_bit_rows_that_align_to_8_bytes(lmh, rows, H, N, R, L, dtype):
    c = _case(rows, H, N, R, L, dtype, dtype, seed=N, ranks=True)
    want = _run(lmh, c)
    _check(c, want)
    wide = torch.full((rows, N + 8), 7.0, dtype=dtype, device="cuda")
    wide[:, 4:N + 4] = c["y"]
    _run(lmh, dict(c, y=wide[:, 4:N + 4]), out=wide[:, 4:N + 4])  # in place, 8 bytes into a row
    assert torch.equal(wide[:, 4:N + 4], want)
    assert (wide[:, :4] == 7).all() and (wide[:, N + 4:] == 7).all()
