"""Which memory the states of a RowStates may have in common: none that is written, but a state's own in place."""
import itertools
import random

import pytest
import torch


@pytest.fixture(scope="module")
def mod():
    from top_reduction_gb300 import lmh
    return lmh


def _bytes(t):
    """The addresses of a tensor's bytes, with repeats."""
    es = t.element_size()
    return [t.data_ptr() + es * sum(i * s for i, s in zip(at, t.stride())) + b
            for at in itertools.product(*(range(n) for n in t.shape)) for b in range(es)]


BASE = torch.zeros(12, 4, 2, 16)
FLAT = torch.zeros(400, dtype=torch.int16)


@pytest.mark.parametrize("tensors,dims,outs", [
    ([BASE[:-1]], 0, [BASE[1:]]),                                     # rows further on
    ([BASE[:4]], 0, [BASE[3:7]]),
    ([BASE[:4], BASE[3:7]], 0, None),                                 # two states in place that share a row
    ([BASE[:, 0], BASE[:, 0, 0]], 0, None),                           # one inside another
    ([BASE[..., :9], BASE[..., 8:]], 0, None),                        # columns that overlap by one
    ([BASE[:6], torch.zeros(6, 4, 2, 16)], 0, [torch.zeros(6, 4, 2, 16), BASE[5:11]]),  # written and read by two
    ([FLAT[:96].view(8, 12)], 0, [FLAT.as_strided((8, 12), (16, 1), 64)]),
    ([FLAT[:20].view(4, 5)], 0, [FLAT[100:].as_strided((4, 5), (3, 1))]),    # an output's own rows overlap
    ([FLAT.as_strided((4, 5), (3, 1))], 0, None),
    ([FLAT.as_strided((5, 4), (1, 3))], 0, [FLAT.as_strided((5, 4), (4, 1), 1)])])
def test_memory_that_is_shared_is_refused(mod, tensors, dims, outs):
    with pytest.raises(ValueError, match="share memory|written twice"):
        mod.RowStates(tensors, dims, None, outs)


@pytest.mark.parametrize("tensors,dims,outs", [
    ([BASE[:6]], 0, [BASE[6:]]), ([BASE[:, 0], BASE[:, 1], BASE[:, 2]], 0, None), ([BASE[:, :, 0], BASE[:, :, 1]], 0, None),
    ([BASE[..., :8], BASE[..., 8:]], 0, None), ([BASE[::2], BASE[1::2]], 0, None), ([BASE[::2]], 0, [BASE[1::2]]),
    ([BASE[..., 3], BASE[..., 4]], 0, None), ([BASE.transpose(0, 1)[0], BASE.transpose(0, 1)[1]], 0, None),
    ([BASE[:4], BASE[:4]], 0, [BASE[4:8], BASE[8:]]),                  # read by two states
    ([BASE[:4, :, :, :1].expand(4, 4, 2, 16)], 0, [BASE[4:8]]),        # read at a stride of 0
    ([FLAT[:21].view(7, 3)], 0, [FLAT.as_strided((7, 3), (5, 2), 100)]),
    ([BASE, torch.zeros(12, 0)], 0, None)])
def test_memory_that_is_apart_is_taken(mod, tensors, dims, outs):
    assert mod.RowStates(tensors, dims, None, outs).rows == tensors[0].shape[0]


def test_layouts_against_their_bytes(mod):
    rng = random.Random(3)
    seen = [0, 0, 0, 0]
    for _ in range(3000):
        def view():
            n = rng.randint(1, 3)
            shape = [rng.randint(1, 4) for _ in range(n)]
            return FLAT.as_strided(shape, [rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24]) for _ in range(n)], rng.randint(0, 60))
        t, u = view(), view()
        a, b = _bytes(t), _bytes(u)
        shared = bool(set(a) & set(b))
        assert mod._meet(mod._layout(t), mod._layout(u), u.data_ptr() - t.data_ptr(), [10 ** 6]) == shared
        own = len(set(a)) < len(a)
        assert mod._meets_itself(t) == own
        seen[shared] += 1
        seen[2 + own] += 1
    assert min(seen) > 300


def test_many_views_of_one_buffer(mod):
    """Sixty layers' caches in one tensor, keys and values interleaved: told apart without looking at every byte."""
    kv = torch.zeros(6, 60, 2, 3, 8, 4)
    steps = []
    meet = mod._meet
    states = mod.RowStates([kv[:, i, j] for i in range(60) for j in range(2)], 0, 2)
    assert states.rows == 6
    for i, j in ((0, 1), (0, 59), (31, 30)):
        left = [mod._MEET_STEPS]
        assert not meet(mod._layout(kv[:, i, 0]), mod._layout(kv[:, j, 1]),
                        kv[:, j, 1].data_ptr() - kv[:, i, 0].data_ptr(), left)
        steps.append(mod._MEET_STEPS - left[0])
    assert max(steps) < 50
