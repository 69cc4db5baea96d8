"""Pages and lengths that are out of range (needs a B200).  In a cache with
positions a row and its position move together, or neither does."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import Store  # noqa: E402
from tests.test_gpu_row_moves import Model, commit, fork  # noqa: E402
from tests.test_gpu_tree_attention import Drafts  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("hkv", [2, 8])
@pytest.mark.parametrize("bad_id", [-1, 1 << 30])
@pytest.mark.parametrize("page", [1, 2, 3])
def test_commit_moves_a_position_only_with_its_row(page, bad_id, hkv):
    # committed rows 0 .. 27, drafted 28 .. 59 (pages 1, 2 and 3 of 16 rows)
    path = [0, 1, 3, 4, 9, 17, 20, 30, 31]
    st = Store(T, 2, 8, hkv, [28, 28], 64, block=16, seed=31, positions=True)
    try:
        st.table[0, page] = bad_id
        m = Model(st)
        ws = commit(st, [path, path])
        for s in range(2):
            for layer in range(2):
                for j, a in enumerate(path):
                    if s == 1 or page not in ((28 + a) // 16, (28 + j) // 16):
                        m.move(layer, s, 28 + a, s, 28 + j)
                        m.move_pos(layer, s, 28 + a, s, 28 + j)
            m.lens[s] += len(path)
        m.same()
        assert T.tria_read_device_status(ws) == 1
    finally:
        st.free()


@pytest.mark.parametrize("hkv", [2, 8])
@pytest.mark.parametrize("bad_id", [-1, 1 << 30])
@pytest.mark.parametrize("who", ["source", "destination"])
def test_fork_copies_a_position_only_with_its_row(who, bad_id, hkv):
    # 40 destinations of 90 rows; block 5 is shared by all but the last two
    n, kids = 90, 40
    st = Store(T, 2, 8, hkv, [n] + [7] * kids, 112, block=16, seed=32, positions=True)
    try:
        st.table[1: kids - 1, 5] = st.table[0, 5]
        bad = [0] if who == "source" else [1, 33, kids]
        for s in bad:
            st.table[s, 2] = bad_id
        m = Model(st)
        assert fork(st, [0] * kids, list(range(1, kids + 1))) == 1
        for s in range(1, kids + 1):
            for layer in range(2):
                for t in range(n):
                    if t // 16 != 2 or (s not in bad and 0 not in bad):
                        m.move(layer, 0, t, s, t)
                        m.move_pos(layer, 0, t, s, t)
            m.lens[s] = n
        m.same()
    finally:
        st.free()


@pytest.mark.parametrize("length", [-1, 129])
@pytest.mark.parametrize("n_seq", [2, 40])
def test_a_bad_length_is_flagged_without_drafted_tokens(length, n_seq):
    st = Store(T, 1, 8, 2, [100] * n_seq, 128, seed=33)
    try:
        d = Drafts(st, 8, [3] * (n_seq - 1) + [0], seed=33)
        d.run()
        assert T.tria_read_device_status(d.ws) == 0
        st.lens[n_seq - 1] = length          # the sequence that has no drafted tokens
        d.run()
        assert T.tria_read_device_status(d.ws) == 1
        d.check(seqs=[0, n_seq - 2])
    finally:
        st.free()
