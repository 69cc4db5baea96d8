"""Arguments of the serving operators that the host looks at alone (no GPU)."""
import pytest

import key_retention_scoring_b200 as T
from key_retention_scoring_b200 import build as tria_build

pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()


def test_wait_limit_refuses_negative_bounds():
    with pytest.raises(T.TriaError) as e:
        T.tria_set_attention_wait_limit(-1)
    assert e.value.status == 1
    T.tria_set_attention_wait_limit(2 ** 63 - 1)
    T.tria_set_attention_wait_limit(0)
