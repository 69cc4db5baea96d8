"""Calls of the cache operators that are refused on the host (a stats handle
needs a GPU; nothing is launched)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import Store  # noqa: E402


@pytest.fixture(scope="module")
def store():
    tria_build.build()
    st = Store(T, 2, 8, 2, [20, 30], 64, block=16, seed=1)
    yield st
    st.free()


def refused(status, call, *args, **kw):
    with pytest.raises(T.TriaError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value


def test_tree_refuses(store):
    st = store
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = q.clone(), torch.zeros((4, 8), device="cuda")
    starts = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    mask = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    ws = T.alloc_workspace(T.tria_tree_workspace_size(st.stats, st.cache, 40))

    def call(layer=0, q=q, starts=starts, most=2, scale=0.1, out=out, ws=ws, **kw):
        T.tria_tree_attention(st.stats, st.cache, layer, q, starts, most, scale, out, ws, **kw)

    for kw in (dict(layer=-1), dict(layer=2), dict(most=0), dict(most=65), dict(scale=0.0), dict(scale=float("nan")),
               dict(most=40, mask=mask), dict(q=q.float()), dict(q=q[:, :4]), dict(q=q[:, :, :64]), dict(q=q[:2]),
               dict(out=out.float()), dict(out=out.transpose(0, 1).contiguous().transpose(0, 1)),
               dict(starts=starts[:2]), dict(starts=starts.long()), dict(lse=lse[:, :4]), dict(lse=lse.double()),
               dict(mask=mask[:2]), dict(mask=mask.float()), dict(starts=starts.cpu()), dict(q=q.cpu())):
        refused(1, call, **kw)
    refused(3, call, ws=ws[256:512][:255])
    refused(3, call, ws=ws[:128])
    refused(1, T.tria_tree_workspace_size, st.stats, st.cache, 0)
    refused(1, T.tria_tree_workspace_size, st.stats, st.cache, 65)
    assert bool((out == 0).all())


def test_commit_refuses(store):
    st = store
    acc = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    cnt = torch.zeros((2,), dtype=torch.int32, device="cuda")
    ws = T.alloc_workspace(T.tria_commit_workspace_size(st.stats, st.cache))

    def call(acc=acc, cnt=cnt, a=0, b=2, ws=ws):
        T.tria_tree_commit(st.stats, st.cache, acc, cnt, a, b, ws)

    for kw in (dict(a=-1), dict(a=1, b=1), dict(b=3), dict(acc=acc[:1]), dict(cnt=cnt[:1]), dict(acc=acc.long()),
               dict(acc=acc[:, :0].contiguous()), dict(acc=acc.cpu()), dict(acc=acc.T.contiguous().T)):
        refused(1, call, **kw)
    refused(3, call, ws=ws[:256])


def test_fork_refuses(store):
    st = store
    ws = T.alloc_workspace(T.tria_fork_workspace_size(st.stats, st.cache))

    def call(src, dst, a=0, b=2, ws=ws):
        T.tria_fork_sequences(st.stats, st.cache, src, dst, a, b, ws)

    before = st.k.clone()
    for src, dst in (([0], [0]), ([0], [2]), ([-1], [1]), ([2], [1]), ([0, 0], [1, 1]), ([0, 1], [1, 0]), ([0, 0], [1])):
        refused(1, call, src, dst)
    refused(1, call, [0], [1], 1, 1)
    refused(1, call, [0], [1], 0, 3)
    refused(3, call, [0], [1], ws=ws[:128])
    call([], [])
    assert torch.equal(before, st.k)
