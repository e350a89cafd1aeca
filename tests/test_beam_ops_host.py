"""Refusals of the adapters', beams' and states' entry points: bad arguments return a status before any
device is touched, and the binding's own checks of tensors."""
import contextlib
import ctypes
import types

import pytest
import torch

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3
A = 1 << 20  # a 256-byte aligned stand-in for a device pointer; nothing is read through it


@pytest.fixture(scope="module")
def mod():
    from top_reduction_gb300 import _build, lmh
    _build.build()
    lmh.load()
    return lmh


def adapters(mod, **change):
    f = dict(down=A, down_adapter_stride=16 * 64, down_row_stride=64, up=A, up_adapter_stride=100 * 16,
             up_row_stride=16, dtype=0, scales=None, ranks=None, count=3, rank=16, H=64, N=100)
    f.update(change)
    return mod.AdaptersArg(**f)


def add(mod, table=None, **change):
    a = dict(x=A, stride=64, tokens=4, idx=None, rows=4, adapter=A, y=A, ys=100, out=2 * A, od=2, os=100, ws=A,
             wb=1 << 30)
    a.update(change)
    t = adapters(mod) if table is None else table
    return mod.load().lmh_add_adapters(a["x"], a["stride"], a["tokens"], a["idx"], a["rows"], a["adapter"], t, a["y"],
                                       a["ys"], a["out"], a["od"], a["os"], a["ws"], a["wb"], None, None)


@pytest.mark.parametrize("change,status", [
    (dict(down=None), INVALID), (dict(up=None), INVALID), (dict(count=0), INVALID), (dict(rank=0), INVALID),
    (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(down_row_stride=56), INVALID), (dict(up_row_stride=8), INVALID),
    (dict(down_adapter_stride=-8), INVALID), (dict(up_adapter_stride=-8), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(dtype=7), UNSUPPORTED), (dict(count=4097), UNSUPPORTED), (dict(rank=136, up_row_stride=136), UNSUPPORTED),
    (dict(rank=12), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(down_row_stride=68), UNSUPPORTED),
    (dict(up_row_stride=20), UNSUPPORTED), (dict(down_adapter_stride=1028), UNSUPPORTED),
    (dict(up_adapter_stride=1604), UNSUPPORTED), (dict(down=A + 8), UNSUPPORTED), (dict(up=A + 2), UNSUPPORTED),
    (dict(H=2147483640, down_row_stride=2147483640), UNSUPPORTED), (dict(N=2147483647), UNSUPPORTED)])
def test_adapter_table_refusals(mod, change, status):
    t = adapters(mod, **change)
    assert add(mod, t) == status
    assert mod.load().lmh_adapters_workspace_bytes(4, t) == 0


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(adapter=None), INVALID), (dict(y=None), INVALID), (dict(out=None), INVALID),
    (dict(rows=-1), INVALID), (dict(tokens=-1), INVALID), (dict(rows=5), INVALID), (dict(stride=63), INVALID),
    (dict(ys=99), INVALID), (dict(os=99), INVALID), (dict(out=A, os=104), INVALID), (dict(ws=None), INVALID),
    (dict(ws=A + 128), INVALID), (dict(od=1), UNSUPPORTED), (dict(od=5), UNSUPPORTED), (dict(x=A + 1), UNSUPPORTED),
    (dict(y=A + 2), UNSUPPORTED), (dict(out=A + 2), UNSUPPORTED)])
def test_add_adapters_refusals(mod, change, status):
    assert add(mod, **change) == status


def beams(mod, **change):
    f = dict(groups=2, beams=4, k=4, keep_slots=0, scores=A, finished=None, pad_id=0, out_scores=2 * A, out_parents=A,
             out_tokens=A)
    f.update(change)
    return mod.BeamsArg(**f)


def select(mod, b, **change):
    a = dict(logits=A, dtype=0, V=1000, stride=1000, mask=None, words=0, ws=A, wb=1 << 30)
    a.update(change)
    return mod.load().lmh_beam_select(b, a["logits"], a["dtype"], a["V"], a["stride"], a["mask"], a["words"], a["ws"],
                                      a["wb"], None, None)


@pytest.mark.parametrize("change,status", [
    (dict(groups=-1), INVALID), (dict(beams=0), INVALID), (dict(k=0), INVALID), (dict(beams=129), UNSUPPORTED),
    (dict(k=129), UNSUPPORTED), (dict(keep_slots=2), INVALID), (dict(keep_slots=1, k=8), INVALID),
    (dict(scores=None), INVALID), (dict(out_scores=None), INVALID), (dict(out_parents=None), INVALID),
    (dict(out_tokens=None), INVALID), (dict(out_scores=A), INVALID), (dict(groups=1 << 30), UNSUPPORTED)])
def test_beam_refusals(mod, change, status):
    b = beams(mod, **change)
    assert select(mod, b) == status
    assert mod.load().lmh_beam_select_lists(b, A, A, 10, None, None) == status
    assert mod.load().lmh_beam_select_lists(None, A, A, 10, None, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(V=0), INVALID), (dict(stride=999), INVALID), (dict(dtype=3), INVALID), (dict(logits=None), INVALID),
    (dict(mask=A, words=31), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 64), INVALID),
    (dict(wb=100), TOO_SMALL), (dict(logits=A + 1), UNSUPPORTED), (dict(logits=A + 2, dtype=2), UNSUPPORTED),
    (dict(V=1 << 29, stride=1 << 29), UNSUPPORTED)])
def test_beam_logits_refusals(mod, change, status):
    assert select(mod, beams(mod), **change) == status


@pytest.mark.parametrize("change,status", [(dict(n=0), INVALID), (dict(ids=None), INVALID), (dict(lps=None), INVALID),
                                           (dict(n=1 << 29), UNSUPPORTED)])
def test_beam_list_refusals(mod, change, status):
    a = dict(ids=A, lps=A, n=10)
    a.update(change)
    assert mod.load().lmh_beam_select_lists(beams(mod), a["ids"], a["lps"], a["n"], None, None) == status


def state(mod, **change):
    two = ctypes.c_int64 * 2
    f = dict(src=A, dst=2 * A, src_row_bytes=64, dst_row_bytes=64, src_outer_bytes=two(0, 0),
             dst_outer_bytes=two(0, 0), n0=1, n1=1, chunk_bytes=64, position_bytes=0)
    f.update({k: two(*v) if isinstance(v, tuple) else v for k, v in change.items()})
    return (mod.RowStateArg * 1)(mod.RowStateArg(**f))


@pytest.mark.parametrize("change,status", [
    (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(n0=-1), INVALID), (dict(n1=-1), INVALID),
    (dict(chunk_bytes=-1), INVALID), (dict(position_bytes=-4), INVALID), (dict(src_row_bytes=-64), INVALID),
    (dict(dst_row_bytes=-64), INVALID), (dict(src_outer_bytes=(0, -1)), INVALID),
    (dict(dst_outer_bytes=(-1, 0)), INVALID), (dict(dst=A, dst_row_bytes=128), INVALID),
    (dict(dst=A, dst_outer_bytes=(64, 0)), INVALID), (dict(chunk_bytes=1 << 42), UNSUPPORTED),
    (dict(n0=1 << 20, n1=1 << 20), UNSUPPORTED)])
def test_state_refusals(mod, change, status):
    assert mod.load().lmh_reorder_rows(state(mod, **change), 1, 2, 4, A, None, None, None) == status


@pytest.mark.parametrize("n,groups,beams_,parents,status", [
    (-1, 2, 4, A, INVALID), (1, -1, 4, A, INVALID), (1, 2, 0, A, INVALID), (1, 2, 129, A, UNSUPPORTED),
    (1, 1 << 30, 4, A, UNSUPPORTED), (1, 2, 4, None, INVALID)])
def test_reorder_refusals(mod, n, groups, beams_, parents, status):
    assert mod.load().lmh_reorder_rows(state(mod), n, groups, beams_, parents, None, None, None) == status
    assert mod.load().lmh_reorder_rows(None, 1, 2, 4, A, None, None, None) == INVALID


def test_no_rows_is_no_work(mod):
    assert add(mod, rows=0, x=None, y=None, out=None, adapter=None, ws=None) == 0
    b = beams(mod, groups=0, scores=None, out_scores=None, out_parents=None, out_tokens=None)
    assert select(mod, b, logits=None, ws=None) == 0
    assert mod.load().lmh_beam_select_lists(b, None, None, 10, None, None) == 0
    assert mod.load().lmh_reorder_rows(state(mod), 1, 0, 4, None, None, None, None) == 0
    assert mod.load().lmh_reorder_rows(None, 0, 2, 4, None, None, None, None) == 0


@pytest.mark.parametrize("groups,beams_,V,some", [(2, 4, 1000, True), (0, 4, 1000, True), (2, 4, 0, False),
                                                  (2, 0, 10, False), (-1, 4, 10, False), (2, 129, 10, False),
                                                  (1, 4, 1 << 29, False), (1 << 30, 4, 10, False)])
def test_beam_workspace(mod, groups, beams_, V, some):
    assert (mod.load().lmh_beam_workspace_bytes(groups, beams_, V) > 0) == some


# ---------------------------------------------------------------------------
# the binding's description of states
# ---------------------------------------------------------------------------

def _rows_of(arg, base, r):
    """The byte offsets from `base` of a row's chunks, as the kernels take them."""
    return [arg.src - base + r * arg.src_row_bytes + i * arg.src_outer_bytes[0] + j * arg.src_outer_bytes[1]
            for i in range(arg.n0) for j in range(arg.n1)]


@pytest.mark.parametrize("shape,dim,along,chunk,chunks", [
    ((6, 10), 0, None, 10, 1), ((6, 10), 0, 1, 10, 1), ((6,), 0, None, 1, 1), ((3, 6, 5), 1, None, 5, 3),
    ((2, 2, 6, 3, 8, 4), 2, 4, 32, 12), ((2, 6, 3, 8, 4), 1, None, 96, 2), ((2, 6, 8, 3, 4), 1, 2, 96, 2),
    ((6, 3, 8, 4), 0, 2, 32, 3)])
def test_rows_of_a_state(mod, shape, dim, along, chunk, chunks):
    t = torch.arange(torch.Size(shape).numel(), dtype=torch.int32).view(shape)
    arg, rows = mod._row_state(t, t, dim, along)
    assert rows == 6 and arg.chunk_bytes == 4 * chunk and arg.n0 * arg.n1 == chunks
    assert arg.position_bytes == (0 if along is None else 4 * chunk // shape[along])
    for r in range(6):
        got = [o // 4 + c for o in _rows_of(arg, t.data_ptr(), r) for c in range(chunk)]
        assert got == t.select(dim, r).flatten().tolist()


def test_rows_of_a_view(mod):
    whole = torch.arange(2 * 2 * 6 * 3 * 8 * 4, dtype=torch.int32).view(2, 2, 6, 3, 8, 4)
    keys = whole[:, 0, :, :, :5]  # the first five of eight positions of one of two
    arg, rows = mod._row_state(keys, torch.empty_like(keys), 1, 3)
    assert (rows, arg.n0, arg.n1, arg.chunk_bytes, arg.position_bytes) == (6, 2, 3, 80, 16)
    for r in range(6):
        got = [o // 4 + c for o in _rows_of(arg, whole.data_ptr(), r) for c in range(20)]
        assert got == keys[:, r].flatten().tolist()


@pytest.mark.parametrize("t,dim,along,what", [
    (torch.zeros(4, 8, 2).transpose(1, 2), 0, 1, "positions must be contiguous"),
    (torch.zeros(4, 8, 2), 1, 0, "must come after"), (torch.zeros(4, 8), 2, None, "no dimension 2"),
    (torch.zeros(4, 1, 1).expand(4, 3, 1), 0, None, "share memory"), (torch.zeros(1, 4).expand(3, 4), 0, None, "share"),
    (torch.zeros(2, 3, 9, 3, 9, 3, 9, 2)[:, :, :2, :, :2, :, :2], 0, None, "two runs")])
def test_states_that_are_refused(mod, t, dim, along, what):
    with pytest.raises(ValueError, match=what):
        mod._row_state(t, t, dim, along)


def test_state_outputs_and_lists_are_checked(mod):
    a, b = torch.zeros(4, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="shape, type and device"):
        mod._row_state(a, torch.zeros(4, 9), 0, None)
    for args, what in (([[]], "no states"), ([[a, torch.zeros(5, 2)]], "4 and 5 rows"), ([[a, a]], "written twice"),
                       ([[a, b], 0, None, [b, torch.zeros(4, 8)]], "written and read"),
                       ([[a], [0, 1]], "one entry"), ([[a], 0, [1, 1]], "one entry")):
        with pytest.raises(ValueError, match=what):
            mod.RowStates(*args)
    assert mod.RowStates([a, b]).rows == 4
    assert mod.RowStates([torch.zeros(4, 0), torch.zeros(4, 2)])._arg[0].chunk_bytes == 0


class _OnGpu1:
    """Stands in for a tensor of a second GPU: the calls look no further before they change device."""
    device = torch.device("cuda", 1)


class _Entered(Exception):
    pass


@pytest.mark.parametrize("call", [
    lambda m: m.add_adapters(_OnGpu1, None, None, None), lambda m: m.beam_select(_OnGpu1, None, 4),
    lambda m: m.beam_select_lists(_OnGpu1, None, None, 4),
    lambda m: m.reorder_rows(_states_on_gpu1(m), None, 4)])
def test_the_tensors_device_is_made_current(mod, call, monkeypatch):
    @contextlib.contextmanager
    def device(d):
        assert d == _OnGpu1.device
        raise _Entered
        yield
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    with pytest.raises(_Entered):
        call(mod)
    with pytest.raises(ValueError, match="stream is of cuda:0"):
        monkeypatch.setattr(mod, "_other_device", lambda d: False)
        stream = types.SimpleNamespace(device=torch.device("cuda", 0))
        {0: lambda: mod.beam_select(_OnGpu1, None, 4, stream=stream)}[0]()


def _states_on_gpu1(m):
    s = m.RowStates([torch.zeros(4, 2)])
    s.device = _OnGpu1.device
    return s


def test_parents_in_a_state_are_refused(mod, monkeypatch):
    t = torch.zeros(8, 4, dtype=torch.int32)
    monkeypatch.setattr(mod, "_other_device", lambda d: False)
    with pytest.raises(ValueError, match="may not lie in a state"):
        mod.reorder_rows([t], t.view(-1)[:8], 4)
    with pytest.raises(ValueError, match="may not lie in a state"):
        mod.reorder_rows([t], torch.zeros(8, dtype=torch.int32), 4, lengths=t.view(-1)[24:])
    with pytest.raises(ValueError, match="whole groups"):
        mod.reorder_rows([t], torch.zeros(8, dtype=torch.int32), 3)


# ---------------------------------------------------------------------------
# the largest sizes, and workspaces that are kept
# ---------------------------------------------------------------------------

def test_sizes_that_32_bits_cannot_go_through_are_refused(mod):
    most = 2147483647 - 65536
    lib = mod.load()
    t = adapters(mod, N=1)
    assert lib.lmh_adapters_workspace_bytes(most + 1, t) == 0
    assert add(mod, t, rows=most + 1, tokens=2147483647) == UNSUPPORTED
    for V in (most + 1, 2147483647):
        b = beams(mod, beams=1, k=1)
        assert lib.lmh_beam_workspace_bytes(2, 1, V) == 0
        assert select(mod, b, V=V, stride=V) == UNSUPPORTED
        assert lib.lmh_beam_select_lists(b, A, A, V, None, None) == UNSUPPORTED
    assert lib.lmh_beam_workspace_bytes(2, 1, most) > 0
    # a length times a position's bytes stays below 2^62
    assert lib.lmh_reorder_rows(state(mod, chunk_bytes=1 << 33, position_bytes=1 << 31, src_row_bytes=1 << 33,
                                      dst_row_bytes=1 << 33), 1, 2, 4, A, A, None, None) == UNSUPPORTED


def test_kept_workspaces_are_a_threads_own(mod, monkeypatch):
    """Two host threads that call on one stream: their kernels may come in turn, so their workspaces differ."""
    import threading
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)
    monkeypatch.setattr(mod, "_SCRATCH", threading.local())
    dev, got = torch.device("cpu"), []
    mine = mod._scratch(1000, dev, 7)
    assert mod._scratch(900, dev, 7) is mine and mod._scratch(900, dev, 8) is not mine
    other = threading.Thread(target=lambda: got.append(mod._scratch(1000, dev, 7)))
    other.start()
    other.join()
    assert got[0].data_ptr() != mine.data_ptr()
    assert mod._scratch(mine.numel() + 1, dev, 7).numel() > mine.numel()
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True)
    assert mod._scratch(1000, dev, 7).data_ptr() not in (mine.data_ptr(), got[0].data_ptr())


def test_misaligned_mask_is_refused(mod):
    assert select(mod, beams(mod), mask=A + 2, words=32) == UNSUPPORTED
