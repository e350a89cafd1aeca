"""Refusals of the decode-step entry points: bad arguments return a status before any device is touched."""
import ctypes

import pytest

INVALID, UNSUPPORTED = 1, 2
A = 1 << 20  # a 16-byte aligned stand-in for a device pointer; nothing is read through it


@pytest.fixture(scope="module")
def mod():
    from top_reduction_gb300 import _build, lmh
    _build.build()
    lmh.load()
    return lmh


def sample(mod, logits=A, dtype=0, rows=2, V=100, stride=100, filters=None, uniforms=A, ids=A):
    f = None if filters is None else ctypes.byref(mod.Filters(**filters))
    return mod.load().lmh_sample_from_logits(logits, dtype, rows, V, stride, f, uniforms, ids, None, None, None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INVALID), (dict(uniforms=None), INVALID), (dict(ids=None), INVALID), (dict(rows=-1), INVALID),
    (dict(V=0), INVALID), (dict(stride=99), INVALID), (dict(dtype=3), INVALID),
    (dict(filters=dict(allowed_mask=A, mask_words=3)), INVALID), (dict(logits=A + 1), UNSUPPORTED),
    (dict(logits=A + 2, dtype=2), UNSUPPORTED), (dict(V=393217, stride=393217), UNSUPPORTED)])
def test_sample_refusals(mod, change, status):
    assert sample(mod, **change) == status


def test_no_rows_is_no_work(mod):
    assert sample(mod, rows=0, logits=None, uniforms=None, ids=None) == 0
    t = table(mod)
    assert mod.load().lmh_project_q4(None, 0, 64, 0, None, 0, t, 1.0, None, 2, 10, None, None) == 0
    assert mod.load().lmh_lookup_q4(None, 0, t, 1.0, None, 0, 64, None, None) == 0


def table(mod, **change):
    f = dict(packed=A, packed_row_bytes=32, scales=A, scale_dtype=0, scale_row_stride=1, zeros=None,
             zero_row_stride=0, V=10, H=64, group=64)
    f.update(change)
    return ctypes.byref(mod.Q4TableArg(**f))


BAD_TABLES = [(dict(packed=None), INVALID), (dict(scales=None), INVALID), (dict(V=0), INVALID), (dict(H=0), INVALID),
              (dict(scale_dtype=9), INVALID), (dict(group=48), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
              (dict(H=96), INVALID), (dict(packed_row_bytes=16), INVALID), (dict(scale_row_stride=0), INVALID),
              (dict(zeros=A, zero_row_stride=0), INVALID), (dict(packed=A + 8), UNSUPPORTED),
              (dict(packed_row_bytes=40), UNSUPPORTED), (dict(scales=A + 1), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", BAD_TABLES)
def test_table_refusals(mod, change, status):
    lib, t = mod.load(), table(mod, **change)
    assert lib.lmh_quantize_q4(A, 64, t, None) == status
    assert lib.lmh_project_q4(A, 0, 64, 1, None, 1, t, 1.0, A, 2, 10, None, None) == status
    assert lib.lmh_lookup_q4(A, 1, t, 1.0, A, 0, 64, None, None) == status


def test_null_table(mod):
    assert mod.load().lmh_lookup_q4(A, 1, None, 1.0, A, 0, 64, None, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(hidden=None), INVALID), (dict(out=None), INVALID), (dict(stride=63), INVALID), (dict(ostride=9), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=5), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(hd=2), UNSUPPORTED), (dict(od=1), UNSUPPORTED), (dict(hidden=A + 1), UNSUPPORTED),
    (dict(out=A + 2), UNSUPPORTED)])
def test_project_refusals(mod, change, status):
    a = dict(hidden=A, hd=0, stride=64, tokens=4, rows=2, scale=1.0, out=A, od=2, ostride=10)
    a.update(change)
    assert mod.load().lmh_project_q4(a["hidden"], a["hd"], a["stride"], a["tokens"], None, a["rows"], table(mod),
                                     a["scale"], a["out"], a["od"], a["ostride"], None, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(ids=None), INVALID), (dict(out=None), INVALID), (dict(n=-1), INVALID), (dict(ostride=63), INVALID),
    (dict(od=7), INVALID), (dict(scale=float("inf")), INVALID), (dict(out=A + 1), UNSUPPORTED)])
def test_lookup_refusals(mod, change, status):
    a = dict(ids=A, n=3, scale=1.0, out=A, od=0, ostride=64)
    a.update(change)
    assert mod.load().lmh_lookup_q4(a["ids"], a["n"], table(mod), a["scale"], a["out"], a["od"], a["ostride"], None,
                                    None) == status


@pytest.mark.parametrize("change,status", [(dict(W=None), INVALID), (dict(stride=63), INVALID),
                                           (dict(W=A + 1), UNSUPPORTED)])
def test_quantise_refusals(mod, change, status):
    a = dict(W=A, stride=64)
    a.update(change)
    assert mod.load().lmh_quantize_q4(a["W"], a["stride"], table(mod), None) == status
