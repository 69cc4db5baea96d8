"""tria_prompt_attention on the GPU against the plain 64-bit form."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import SCALE, attend, causal, check  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


class Prompt:
    """Packed q, k, v of given lengths; `lead` and `tail` rows belong to no sequence."""

    def __init__(self, hq, hkv, lens, seed=0, lead=0, tail=0, form="plain", sigma=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.lens, self.lead = hq, hkv, lens, lead
        self.n = n = lead + sum(lens) + tail
        mk = lambda h, s=1.0: (s * torch.randn((n, h, 128), generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
        q, k, v = mk(hq, sigma), mk(hkv, sigma), mk(hkv)
        if form == "fused":       # slices of one projection
            f = torch.cat([q, k, v], 1)
            q, k, v = f[:, :hq], f[:, hq: hq + hkv], f[:, hq + hkv:]
        elif form == "heads":     # [heads][tokens][128], and rows with a gap
            q = q.transpose(0, 1).contiguous().transpose(0, 1)
            k = k.transpose(0, 1).contiguous().transpose(0, 1)
            w = torch.zeros((n, hkv, 200), dtype=torch.bfloat16, device="cuda")
            w[:, :, :128] = v
            v = w[:, :, :128]
        self.q, self.k, self.v = q, k, v
        at, s = lead, [lead]
        for x in lens:
            at += x
            s.append(at)
        self.starts = torch.tensor(s, dtype=torch.int32, device="cuda")
        self.desc = T.model_desc(1, hq, hkv, T.PAIR_NEOX, 1e4)
        self.ws = T.alloc_workspace(T.tria_prompt_workspace_size(self.desc, len(lens)))
        self.out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, hq), 7.0, device="cuda")

    def run(self, scale=SCALE, stream=None, lse=True):
        T.tria_prompt_attention(self.desc, self.q, self.k, self.v, self.starts, scale, self.out, self.ws,
                                lse=self.lse if lse else None, stream=stream)

    def check(self, scale=SCALE, seqs=None, heads=None, lse=True):
        g = self.hq // self.hkv
        starts = self.starts.tolist()
        for s in seqs if seqs is not None else range(len(self.lens)):
            a, b = starts[s], starts[s + 1]
            if a == b:
                continue
            for h in heads if heads is not None else range(self.hq):
                ref = attend(self.q[a:b, h], self.k[a:b, h // g], self.v[a:b, h // g], causal(b - a), scale)
                check(self.out[a:b, h], self.lse[a:b, h] if lse else None, ref, f"seq {s} head {h}")

    def untouched(self):
        """Rows of no sequence keep what they held."""
        a, b = self.lead, self.lead + sum(self.lens)
        for x in (self.out, self.lse):
            assert bool((x[:a] == 7.0).all()) and bool((x[b:] == 7.0).all())


HEADS = [(2, 2), (4, 2), (8, 2), (16, 2), (16, 1)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [127, 128, 129], [0, 5, 0, 300, 0], [257, 31, 64, 513]],
                         ids=lambda x: "-".join(map(str, x)))
def test_matches_the_plain_form(hq, hkv, lens):
    p = Prompt(hq, hkv, lens, seed=len(lens) + hq, lead=3, tail=5)
    p.run()
    p.check()
    p.untouched()
    assert T.tria_read_device_status(p.ws) == 0


@pytest.mark.parametrize("form", ["fused", "heads"])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (16, 1)])
def test_strided_inputs(form, hq, hkv):
    p = Prompt(hq, hkv, [200, 77], seed=3, form=form)
    p.run()
    p.check(heads=[0, 1, hq - 1])


def test_without_lse_writes_the_same_rows():
    p = Prompt(8, 2, [300, 40], seed=4)
    p.run()
    a = p.out.clone()
    p.out.fill_(7.0)
    p.lse.fill_(7.0)
    p.run(lse=False)
    assert torch.equal(a, p.out) and bool((p.lse == 7.0).all())


@pytest.mark.parametrize("scale,sigma", [(SCALE, 6.0), (1e-6, 1.0), (3.0, 1.0)])
def test_logits_small_and_large(scale, sigma):
    # sigma 6: logits of +-36 sqrt(128) scale, a few keys hold all the weight
    p = Prompt(8, 2, [400], seed=5, sigma=sigma)
    p.run(scale=scale)
    p.check(scale=scale)


def test_growing_logits_move_the_running_maximum():
    # each key's logit exceeds all before it, so the maximum moves at every tile
    p = Prompt(4, 1, [900], seed=6)
    r = torch.linspace(0.2, 8.0, 900, device="cuda")[:, None, None]
    p.k.copy_((torch.ones_like(p.k).float() * r).to(torch.bfloat16))
    p.q.copy_(torch.ones_like(p.q))
    p.run()
    p.check()


def test_long_prompt():
    p = Prompt(8, 2, [4097], seed=7)
    p.run()
    p.check(heads=[0, 5, 7])


def test_many_short_sequences():
    lens = [(7 * i) % 23 for i in range(300)]
    p = Prompt(8, 2, lens, seed=8)
    p.run()
    p.check(seqs=range(0, 300, 13), heads=[0, 7])
    p.untouched()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_row_does_not_see_does_not_reach_it(hq, hkv, bad):
    p = Prompt(hq, hkv, [150, 90, 200], seed=9, lead=2, tail=4)
    for x in (p.k, p.v):
        x[:2] = bad
        x[-4:] = bad                       # rows of no sequence
        x[2 + 150: 2 + 150 + 90] = bad     # the middle sequence, whole
        x[2 + 240 + 130, :, 5] = bad       # one later token of the last one
    p.q[2 + 150: 2 + 150 + 90] = bad
    p.run()
    p.check(seqs=[0])
    a, g = 2 + 240, hq // hkv
    for h in range(hq):
        ref = attend(p.q[a: a + 130, h], p.k[a: a + 130, h // g], p.v[a: a + 130, h // g], causal(130))
        check(p.out[a: a + 130, h], p.lse[a: a + 130, h], ref, f"before the bad token, head {h}")
    p.untouched()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_no_number_reaches_the_rows_that_see_it(bad):
    p = Prompt(8, 2, [300], seed=10)
    p.v[140, 1, 17] = bad
    p.run()
    for h in range(8):
        col = p.out[:, h, 17]
        assert bool(torch.isfinite(col[:140]).all())
        assert bool(torch.isfinite(col[140:]).all()) == (h < 4), h
        assert bool(torch.isfinite(torch.cat([p.out[:, h, :17], p.out[:, h, 18:]], 1)).all())


def test_values_that_are_no_numbers_in_many_short_sequences():
    # several short items for each processor, one after another in either half
    lens = [1 + (37 * i) % 190 for i in range(120)]
    p = Prompt(32, 8, lens, seed=17)
    want = torch.ones(p.out.shape[:2], dtype=torch.bool, device="cuda")  # dim 17 is finite
    at = 0
    for i, n in enumerate(lens):
        j, h = (11 * i) % n, i % 8
        p.v[at + j, h, 17] = [float("inf"), float("-inf"), float("nan")][i % 3]
        want[at + j: at + n, 4 * h: 4 * h + 4] = False
        at += n
    for _ in range(20):
        p.out.fill_(7.0)
        p.run()
        fin = torch.isfinite(p.out)
        assert torch.equal(fin[:, :, 17], want)
        assert bool(fin[:, :, :17].all()) and bool(fin[:, :, 18:].all())


@pytest.mark.parametrize("starts", [[0, 10, 5, 20], [-1, 10, 15, 20], [0, 10, 15, 21]])
def test_bad_starts_are_flagged(starts):
    p = Prompt(8, 2, [10, 5, 5], seed=11)
    p.starts.copy_(torch.tensor(starts, dtype=torch.int32))
    p.run()
    assert T.tria_read_device_status(p.ws) == 1
    ok = [i for i in range(3) if 0 <= starts[i] <= starts[i + 1] <= 20]
    if starts != [0, 10, 5, 20]:
        p.check(seqs=ok)


def test_equal_bits_on_another_stream_and_from_a_graph():
    p = Prompt(32, 8, [700, 3, 150], seed=12)
    p.run()
    a, al = p.out.clone(), p.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.out.fill_(1.0)
    side.wait_stream(torch.cuda.current_stream())
    p.run(stream=side)
    side.synchronize()
    assert torch.equal(a, p.out) and torch.equal(al, p.lse)
    # two graphs over one workspace, replayed in turn
    p2 = Prompt(32, 8, [40, 900], seed=13)
    p2.ws = p.ws
    p2.run()
    b = p2.out.clone()
    graphs = []
    for x in (p, p2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(3):
        p.out.fill_(1.0)
        p2.out.fill_(1.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, p.out) and torch.equal(b, p2.out)
    assert T.tria_read_device_status(p.ws) == 0


def test_no_tokens_is_no_work():
    p = Prompt(8, 2, [0, 0], seed=14)
    p.run()
    assert T.tria_read_device_status(p.ws) == 0


def test_calls_that_read_one_another_between_copies_and_joined_streams():
    # A call's blocks may be resident before the kernel, copy or fill before it has ended.
    lens = [700, 3, 1500]
    p, q = Prompt(8, 8, lens, seed=15), Prompt(8, 8, lens, seed=16)
    keep_q, side = q.q.clone(), torch.cuda.Stream()
    mid = torch.empty_like(p.out)

    def chain(wait):
        main = torch.cuda.current_stream()
        q.q.copy_(keep_q)                       # a copy, then a call that reads it
        q.run()
        wait()
        p.out.zero_()                           # a fill, then a call over it
        T.tria_prompt_attention(p.desc, q.out, p.k, p.v, p.starts, SCALE, p.out, p.ws, lse=p.lse)
        wait()
        T.tria_prompt_attention(p.desc, p.out, q.out, p.out, p.starts, SCALE, mid, p.ws, lse=p.lse)
        wait()
        side.wait_stream(main)                  # two streams, and their join
        with torch.cuda.stream(side):
            T.tria_prompt_attention(p.desc, mid, p.k, p.v, p.starts, SCALE, p.out, p.ws, lse=p.lse)
        T.tria_prompt_attention(q.desc, mid, mid, q.v, q.starts, SCALE, q.out, q.ws, lse=q.lse)
        main.wait_stream(side)
        wait()
        T.tria_prompt_attention(p.desc, q.out, p.out, q.out, p.starts, SCALE, mid, p.ws, lse=p.lse)
        q.q.copy_(mid)                          # a copy that reads the last call's rows

    chain(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = q.q.clone()
    for _ in range(5):
        chain(lambda: None)
        torch.cuda.synchronize()
        assert torch.equal(want, q.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(lambda: None)
    for _ in range(5):
        q.q.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, q.q)
    assert T.tria_read_device_status(p.ws) == 0 and T.tria_read_device_status(q.ws) == 0
