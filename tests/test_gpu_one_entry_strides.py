"""One token or one head of rows whose length is no multiple of 8 elements: the
stride of a dimension of one entry plays no part (needs a B200)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import Store  # noqa: E402
from tests.test_gpu_prompt_attention import Prompt  # noqa: E402
from tests.test_gpu_tree_attention import Drafts  # noqa: E402
import key_retention_scoring_b200 as T  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


def odd(x):
    """x with an odd stride in each of its dimensions of one entry."""
    n, h, _ = x.shape
    if n > 1:
        return x.as_strided(x.shape, (128, 131, 1))
    row = torch.zeros((1, h * 128 + 5), dtype=x.dtype, device=x.device)
    y = row.as_strided(x.shape, (h * 128 + 5, 131 if h == 1 else 128, 1))
    y.copy_(x)
    return y


@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1), (4, 1)])
@pytest.mark.parametrize("n", [1, 40])
def test_prompt(n, hq, hkv):
    p = Prompt(hq, hkv, [n], seed=41)
    for name in "qkv":
        x = getattr(p, name)
        if n == 1 or x.shape[1] == 1:
            setattr(p, name, odd(x))
    p.run()
    p.check()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1)])
def test_tree(hq, hkv):
    st = Store(T, 1, hq, hkv, [300], 320, seed=42)
    try:
        d = Drafts(st, hq, [1], seed=42)
        d.q = odd(d.q)
        d.run()
        d.check()
    finally:
        st.free()
