"""Logits of prompt and tree attention at the ends of their range (needs a B200)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import Store, attend, causal, check, draft_sees  # noqa: E402
from tests.test_gpu_prompt_attention import Prompt  # noqa: E402
from tests.test_gpu_tree_attention import Drafts  # noqa: E402

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


def no_softmax(out, lse):
    assert bool(torch.isnan(out.float()).all()) and bool((lse == -INF).all())


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 1)])
def test_prompt_rows_whose_logits_are_all_minus_infinity(hq, hkv):
    lens, rows = [700, 90, 1], [0, 5, 63, 64, 300, 699, 700 + 89, 790]
    p = Prompt(hq, hkv, lens, seed=51)
    p.k[:, :, 0] = 1.0
    p.q[rows, :, 0] = -INF
    p.run()
    no_softmax(p.out[rows], p.lse[rows])
    others = torch.ones(p.n, dtype=torch.bool, device="cuda")
    others[rows] = False
    at = 0
    for n in lens:
        keep = others[at: at + n]
        for h in (0, hq - 1):
            q, k, v = (x[at: at + n, i] for x, i in ((p.q, h), (p.k, h * hkv // hq), (p.v, h * hkv // hq)))
            if bool(keep.any()):
                check(p.out[at: at + n, h][keep], p.lse[at: at + n, h][keep], attend(q[keep], k, v, causal(n)[keep]), h)
        at += n
    assert T.tria_read_device_status(p.ws) == 0


# one block's keys, several blocks' (partials), more than 128 rows, and none committed
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("n_ctx,n_draft", [(40, 5), (20011, 5), (0, 5), (500, 40), (0, 300)])
def test_tree_rows_whose_logits_are_all_minus_infinity(n_ctx, n_draft, block):
    st = Store(T, 1, 16, 2, [n_ctx, 700], max(n_ctx, 700) + n_draft + 3, block=block, seed=52)
    try:
        st.k[..., 0] = 1.0
        d = Drafts(st, 16, [n_draft, 3], seed=52)
        rows = [0, 3, n_draft - 1]
        d.q[rows, :, 0] = -INF
        d.mask[1] = 0                       # sees its committed rows, or nothing
        d.run()
        no_softmax(d.out[rows], d.lse[rows])
        others = [i for i in range(n_draft) if i not in rows]
        sees = draft_sees(n_ctx, n_draft, d.mask[:n_draft])
        for h in (0, 15):
            k, v = (st.rows(x, 0, 0, h // 8, n_ctx + n_draft) for x in (st.k, st.v))
            check(d.out[others, h], d.lse[others, h], attend(d.q[others, h], k, v, sees[others]), h)
        if n_ctx == 0:
            assert bool((d.out[1] == 0).all()) and bool((d.lse[1] == -INF).all())
        d.check(seqs=[1], heads=[0, 15])
    finally:
        st.free()


@pytest.mark.parametrize("n_draft", [5, 40])
def test_keys_whose_logits_are_minus_infinity_have_no_weight(n_draft):
    # whole pieces of the keys, and every second one of the rest
    n = 20011
    st = Store(T, 1, 16, 2, [n], n + n_draft, seed=53)
    try:
        gone = torch.zeros(n + n_draft, dtype=torch.bool, device="cuda")
        gone[:12000] = True
        gone[12000: n: 2] = True
        d = Drafts(st, 16, [n_draft], seed=53)
        d.q[:, :, 0] = 1.0
        st.k[0, 0, :, gone, 0] = -INF
        d.run()
        sees = draft_sees(n, n_draft, d.mask) & ~gone
        for h in (0, 15):
            k, v = (st.rows(x, 0, 0, h // 8, n + n_draft) for x in (st.k, st.v))
            k[gone] = 0.0                   # not seen by the plain form
            check(d.out[:, h], d.lse[:, h], attend(d.q[:, h], k, v, sees), h)
    finally:
        st.free()
