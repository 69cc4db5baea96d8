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


# Logits that are exact in fp32 (products of bf16 numbers in one or two dims), so that
# the tolerance is that of the softmax alone: weights within 2^-8 + 2^-13 (P in bf16,
# the exponential), the output rounded to bf16 (2^-8); lse = RN(RN(max qs) + log2 l) ln 2
# with qs and ln 2 within 2^-25 of theirs and three roundings of 2^-24: within 2^-21.
def far_rows(kind, n, e, sign, gen):
    """[n] and [n] of a key's first two dims, and of a query's, scaled to 2^e."""
    a, b = 2.0 ** (e // 2), 2.0 ** (e - e // 2)
    j = torch.arange(n, device="cuda", dtype=torch.float64)
    zero = torch.zeros(n, device="cuda", dtype=torch.float64)
    if kind == "ties":          # equal to the largest, a step of bf16 below it, far below it
        off = torch.tensor([0, 0, 1, 2, 60], device="cuda")[torch.randint(0, 5, (n,), generator=gen, device="cuda")]
        return b * (sign - 2.0 ** -7 * off), zero, a, 0.0
    if kind == "rising":        # from 1 to 2^e in size, the largest last
        return torch.sort(sign * torch.exp2(j * (e / (n - 1)))).values, zero, 1.0, 0.0
    if kind == "falling":
        return torch.sort(sign * torch.exp2(j * (e / (n - 1))), descending=True).values, zero, 1.0, 0.0
    small = torch.randint(-24, 25, (n,), generator=gen, device="cuda").double() * 0.125   # "near": 2^e and a little
    return sign * b + zero, small, a, 1.0


FAR = [("ties", e, s) for e in (20, 28, 31, 32, 40, 100) for s in (1, -1)] + [
    (k, e, s) for k in ("rising", "falling") for e in (28, 33, 60, 110) for s in (1, -1)] + [("near", 20, 1), ("near", 20, -1)]
LIMIT = 2.0 ** 30 * 0.6931471805599453


def fill_far(k, q, kind, e, sign, seed):
    """k [n, heads, 128], q [m, heads, 128] in place."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k.zero_()
    q.zero_()
    for h in range(k.shape[1]):
        k0, k1, q0, q1 = far_rows(kind, k.shape[0], e, sign, gen)
        k[:, h, 0], k[:, h, 1] = k0.to(k.dtype), k1.to(k.dtype)
    q[:, :, 0], q[:, :, 1] = q0, q1


def check_exact(out, lse, q, k, v, allowed, where):
    """Rows within the range against the formula, the others as they are documented.
    No row's largest logit is so near the range's ends that its roundings decide."""
    z = torch.where(allowed, q.double() @ k.double().T, -INF)
    top = z.amax(1)
    assert not bool(((top.abs() / LIMIT - 1.0).abs() < 2.0 ** -20).any())
    above, below = top > LIMIT, top < -LIMIT
    assert bool(torch.isnan(out[above | below].float()).all())
    assert bool(torch.isnan(lse[above]).all()) and bool((lse[below] == -INF).all())
    z, out, lse = (x[~(above | below)] for x in (z, out, lse))
    if z.shape[0] == 0:
        return
    ref = torch.logsumexp(z, 1)
    w = torch.exp(z - z.amax(1, keepdim=True))
    w = w / w.sum(1, keepdim=True)
    want = w @ v.double()
    moved = (w @ v.double().abs()) * (2.0 ** -8 + 2.0 ** -13)
    d = (out.double() - want).abs()
    assert bool((d <= moved + 2.0 ** -8 * (want.abs() + moved)).all()), (where, float(d.max()))
    assert bool(((lse.double() - ref).abs() <= 2.0 ** -21 * ref.abs() + 2e-5).all()), where


@pytest.mark.parametrize("kind,e,sign", FAR)
def test_prompt_logits_far_from_zero(kind, e, sign):
    p = Prompt(4, 2, [400], seed=54)
    fill_far(p.k, p.q, kind, e, sign, 55)
    p.run(scale=1.0)
    for h in range(4):
        check_exact(p.out[:, h], p.lse[:, h], p.q[:, h], p.k[:, h // 2], p.v[:, h // 2], causal(400), h)


@pytest.mark.parametrize("n_draft", [5, 40])
@pytest.mark.parametrize("kind,e,sign", FAR)
def test_tree_logits_far_from_zero(kind, e, sign, n_draft):
    n = 8000
    st = Store(T, 1, 16, 2, [n], n + n_draft, seed=56)
    try:
        d = Drafts(st, 16, [n_draft], seed=56)
        fill_far(st.k[0, 0].transpose(0, 1), d.q, kind, e, sign, 57)
        d.run(scale=1.0)
        sees = draft_sees(n, n_draft, d.mask)
        for h in (0, 7, 8):
            k, v = (st.rows(x, 0, 0, h // 8, n + n_draft) for x in (st.k, st.v))
            check_exact(d.out[:, h], d.lse[:, h], d.q[:, h], k, v, sees, h)
    finally:
        st.free()
