"""Refusals of the decode-step calls that only the Python binding can see: tensors that the kernels
would write or read in place of what they were given (types, sizes, devices, streams)."""
import contextlib
import types

import pytest
import torch

from top_reduction_gb300 import lmh as L

CPU, CUDA = torch.device("cpu"), torch.device("cuda", 0)


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(4, dtype=torch.int64), lambda: torch.zeros(4, dtype=torch.float32),
    lambda: torch.zeros(3, dtype=torch.int32), lambda: torch.zeros(8, dtype=torch.int32)[::2],
    lambda: torch.zeros(4, dtype=torch.int32, device="meta"), lambda: torch.zeros(4, 2, dtype=torch.int32).t()])
def test_a_written_tensor_is_checked(make):
    with pytest.raises(ValueError, match="ids must be a contiguous int32"):
        L._written(make(), L._WORDS, 4, CPU, "ids")


def test_written_tensors_that_fit():
    for t in (torch.zeros(4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.uint32)):
        assert L._written(t, L._WORDS, 4, CPU, "ids") == t.data_ptr()
    assert L._written(None, L._FLOATS, 4, CPU, "sampled_logprob") is None
    assert L._status_word(None, CPU) is None
    with pytest.raises(ValueError, match="dev_status"):
        L._status_word(torch.zeros(0, dtype=torch.int32), CPU)


def test_stream_of_another_device():
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        L._on_stream(stream, CUDA)


class _OnGpu1:
    """Stands in for a tensor of a second GPU: the calls look no further before they change device."""
    device = torch.device("cuda", 1)
    is_cuda = True
    dtype = torch.bfloat16

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        s = (self.shape[-1], 1)[-len(self.shape):]
        return s if d is None else s[d]

    def is_contiguous(self):
        return True


class _Entered(Exception):
    pass


@pytest.mark.parametrize("call", [
    lambda: L.sample_from_logits(_OnGpu1(2, 100), None), lambda: L.quantize_q4(_OnGpu1(100, 64)),
    lambda: L.project_q4(_OnGpu1(2, 64), types.SimpleNamespace(device=_OnGpu1.device, V=10, H=64)),
    lambda: L.lookup_q4(_Ids(2), types.SimpleNamespace(device=_OnGpu1.device, V=10, H=64))])
def test_the_tensors_device_is_made_current(call, monkeypatch):
    @contextlib.contextmanager
    def device(d):
        assert d == _OnGpu1.device
        raise _Entered
        yield
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    with pytest.raises(_Entered):
        call()


class _Ids(_OnGpu1):
    dtype = torch.int32


# ---------------------------------------------------------------------------
# the calls themselves: refused before anything is launched
# ---------------------------------------------------------------------------

def _draw(lmh, out=None, **more):
    z, u = torch.zeros(4, 100, device="cuda"), torch.rand(4, device="cuda")
    return lmh.sample_from_logits(z, u, out=out, **more)


def _out(ids=None, lps=None):
    return {"sampled_ids": torch.zeros(4, dtype=torch.int32, device="cuda") if ids is None else ids,
            "sampled_logprob": torch.zeros(4, device="cuda") if lps is None else lps}


@pytest.mark.gpu
@pytest.mark.parametrize("out", [
    lambda: _out(ids=torch.zeros(4, dtype=torch.int64, device="cuda")),
    lambda: _out(ids=torch.zeros(3, dtype=torch.int32, device="cuda")),
    lambda: _out(ids=torch.zeros(4, dtype=torch.int32)),
    lambda: _out(ids=torch.zeros(8, dtype=torch.int32, device="cuda")[::2]),
    lambda: _out(lps=torch.zeros(4, dtype=torch.float64, device="cuda")),
    lambda: _out(lps=torch.zeros(2, device="cuda")), lambda: _out(lps=torch.zeros(4))])
def test_draw_refuses_outputs_that_do_not_fit(lmh, out):
    o = out()
    with pytest.raises(ValueError):
        _draw(lmh, o)
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in o.values())


@pytest.mark.gpu
@pytest.mark.parametrize("mask", [lambda: torch.zeros(4, 4, device="cuda"), lambda: torch.zeros(4, 4, dtype=torch.int16),
                                  lambda: torch.zeros(3, 4, dtype=torch.int32), lambda: torch.zeros(16, dtype=torch.int32)])
def test_draw_refuses_masks_that_do_not_fit(lmh, mask):
    with pytest.raises(ValueError, match="mask"):
        _draw(lmh, mask=mask())


@pytest.mark.gpu
def test_draw_takes_larger_outputs_and_no_logprobs(lmh):
    ids = torch.full((6,), -7, dtype=torch.int32, device="cuda")
    _draw(lmh, {"sampled_ids": ids, "sampled_logprob": None})
    assert (ids[:4] >= 0).all() and (ids[4:] == -7).all()


@pytest.mark.gpu
def test_tensors_on_the_host_are_refused(lmh):
    W = torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda")
    t = lmh.quantize_q4(W, 64)
    x, ids = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: lmh.project_q4(x, t, dev_status=bad), lambda: lmh.lookup_q4(ids, t, dev_status=bad),
                 lambda: _draw(lmh, dev_status=bad)):
        with pytest.raises(ValueError, match="dev_status"):
            call()
    for call in (lambda: lmh.project_q4(x, t, row_idx=ids.cpu()), lambda: lmh.project_q4(x.cpu(), t),
                 lambda: lmh.project_q4(x, t, out=torch.zeros(2, 10)), lambda: lmh.lookup_q4(ids.cpu(), t),
                 lambda: lmh.lookup_q4(ids, t, out=torch.zeros(2, 64, dtype=torch.bfloat16))):
        with pytest.raises(AssertionError):
            call()


@pytest.mark.parametrize("change", [dict(V=2 ** 31 - 127), dict(V=2 ** 31 - 1), dict(H=2 ** 31 - 128, stride=2 ** 31),
                                    dict(H=2 ** 31 - 16384 + 128, stride=2 ** 31)])
def test_projection_refuses_sizes_that_32_bits_cannot_round_up(change):
    """Through the C entry; nothing is read through the stand-in pointers."""
    from top_reduction_gb300 import _build
    _build.build()
    a = dict(V=10, H=128, stride=128)
    a.update(change)
    A, H = 1 << 20, a["H"]
    t = L.Q4TableArg(A, H // 2, A, 0, H // 128, None, 0, a["V"], H, 128)
    assert L.load().lmh_project_q4(A, 0, a["stride"], 1, None, 1, t, 1.0, A, 2, a["V"], None, None) == 2
