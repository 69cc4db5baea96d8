"""Calls of the serving operators that are refused on the host, before any CUDA
call: through the C entry points with made-up addresses that nothing reads."""
import ctypes

import pytest

import key_retention_scoring_b200 as T
from key_retention_scoring_b200 import build as tria_build

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x7000000000  # an aligned address


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()


def prompt(desc=None, **kw):
    a = dict(q=A, qt=1024, qh=128, k=A, kt=256, kh=128, v=A, vt=256, vh=128, n=0, starts=A, n_seq=1, scale=0.1, out=A,
             lse=A, ws=A, size=256)
    a.update(kw)
    desc = desc or T.model_desc(1, 8, 2, T.PAIR_NEOX, 1e4)
    return T.lib().tria_prompt_attention(ctypes.byref(desc), *a.values(), None)


def test_prompt_without_tokens_is_fine():
    assert prompt() == OK
    assert prompt(lse=None, q=None, k=None, v=None, out=None) == OK


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(n=2 ** 31), dict(n_seq=0), dict(n_seq=1025), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(starts=None), dict(starts=A + 2), dict(qt=0), dict(qt=-8),
    dict(qt=1020), dict(qh=4), dict(kt=0), dict(kh=-128), dict(vt=12), dict(vh=0), dict(q=A + 8), dict(k=A + 2),
    dict(v=A + 8), dict(out=A + 4), dict(lse=A + 2), dict(n=5, q=None), dict(n=5, k=None), dict(n=5, v=None),
    dict(n=5, out=None)], ids=str)
def test_prompt_refuses(change):
    assert prompt(**change) == INVALID


def test_prompt_refuses_shapes_and_workspaces():
    assert prompt(T.model_desc(1, 6, 2, T.PAIR_NEOX, 1e4)) == UNSUPPORTED      # G = 3
    assert prompt(T.model_desc(1, 64, 2, T.PAIR_NEOX, 1e4)) == UNSUPPORTED     # G = 32
    assert prompt(T.model_desc(1, 8, 2, T.PAIR_NEOX, 1e4, head_dim=64)) == UNSUPPORTED
    assert prompt(T.model_desc(1, 7, 2, T.PAIR_NEOX, 1e4)) == INVALID
    assert prompt(T.model_desc(1, 8, 0, T.PAIR_NEOX, 1e4)) == INVALID
    for change in (dict(ws=None), dict(ws=A + 128), dict(size=255)):
        assert prompt(**change) == WORKSPACE
    size = ctypes.c_size_t()
    d = T.model_desc(1, 8, 2, T.PAIR_NEOX, 1e4)
    assert T.lib().tria_prompt_workspace_size(None, 1, ctypes.byref(size)) == INVALID
    assert T.lib().tria_prompt_workspace_size(ctypes.byref(d), 0, ctypes.byref(size)) == INVALID
    assert T.lib().tria_prompt_workspace_size(ctypes.byref(d), 1, ctypes.byref(size)) == OK and size.value >= 256


def test_cache_operators_refuse_missing_objects():
    lib, size = T.lib(), ctypes.c_size_t()
    view = T.CacheView()
    assert lib.tria_tree_workspace_size(None, ctypes.byref(view), 1, ctypes.byref(size)) == INVALID
    assert lib.tria_commit_workspace_size(None, ctypes.byref(view), ctypes.byref(size)) == INVALID
    assert lib.tria_fork_workspace_size(None, ctypes.byref(view), ctypes.byref(size)) == INVALID
    assert lib.tria_tree_attention(None, ctypes.byref(view), 0, A, 1024, 128, 1, A, 1, None, 0, 0.1, A, None, A, 256,
                                   None) == INVALID
    assert lib.tria_tree_commit(None, ctypes.byref(view), A, A, 1, 0, 1, A, 512, None) == INVALID
    assert lib.tria_fork_sequences(None, ctypes.byref(view), A, A, 0, 0, 1, A, 256, None) == INVALID


def test_binding_refuses_tensors_off_the_device():
    d = T.model_desc(1, 8, 2, T.PAIR_NEOX, 1e4)
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    s = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(T.TriaError) as e:
        T.tria_prompt_attention(d, q, k, k, s, 0.1, q.clone(), torch.zeros(256, dtype=torch.uint8))
    assert e.value.status == INVALID
