"""Arguments of the serving operators that the host looks at alone (no GPU)."""
import ctypes

import numpy as np
import pytest

import key_retention_scoring_b200 as T
from key_retention_scoring_b200 import build as tria_build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()


def test_wait_limit_refuses_negative_bounds():
    with pytest.raises(T.TriaError) as e:
        T.tria_set_attention_wait_limit(-1)
    assert e.value.status == 1
    T.tria_set_attention_wait_limit(2 ** 63 - 1)
    T.tria_set_attention_wait_limit(0)


@pytest.mark.parametrize("shape,strides,want", [
    ((5, 8), (1024, 128, 1), (1024, 128)), ((5, 1), (1024, 77, 1), (1024, 128)), ((1, 8), (1028, 128, 1), (1024, 128)),
    ((1, 8), (3, 256, 1), (2048, 256)), ((1, 1), (1028, 131, 1), (128, 128)), ((0, 8), (0, 128, 1), (1024, 128)),
    ((1, 8), (1028, 4, 1), (32, 4))], ids=str)
def test_strides_of_one_entry_dimensions_are_not_looked_at(shape, strides, want):
    assert T._row_strides(strides, *shape) == want


@pytest.mark.parametrize("x", [[], (), [0, 3], (2,), np.array([1, 2]), np.array([5], np.uint8), torch.tensor([4, 1])], ids=str)
def test_fork_indices(x):
    got = T._indices("here", "src", x)
    assert got.typecode == "i" and got.itemsize == 4 and got.tolist() == [int(v) for v in x]


@pytest.mark.parametrize("x", [[0.9], [2 ** 32 + 1], np.array([2 ** 32 + 1]), np.array([-2 ** 31 - 1]), np.array([2 ** 64 - 1], np.uint64),
                               [[0, 1]], 3, "12", ["1"], [None], torch.tensor([1.0])], ids=str)
def test_fork_refuses_what_is_no_index(x):
    with pytest.raises(T.TriaError) as e:
        T._indices("here", "src", x)
    assert e.value.status == 1


@pytest.mark.parametrize("scale,status", [(2.35e38, 0), (2.4e38, 1), (3.4e38, 1), (1e-45, 0), (0.0, 1)])
def test_the_scale_in_base_2_must_be_a_number(scale, status):
    d, a = T.model_desc(1, 8, 2, T.PAIR_NEOX, 1e4), 0x7000000000
    assert T.lib().tria_prompt_attention(ctypes.byref(d), a, 1024, 128, a, 256, 128, a, 256, 128, 0, a, 1, scale, a, a, a,
                                         256, None) == status
