"""Pages outside the pool, in a cache with positions: a row and its position move
together, or neither does (needs a B200)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import Store  # noqa: E402
from tests.test_gpu_row_moves import Model, commit  # noqa: E402


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
