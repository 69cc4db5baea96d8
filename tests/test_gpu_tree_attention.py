"""tria_tree_attention on the GPU against the plain 64-bit form."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import SCALE, Store, attend, check, draft_sees, tree_bits  # noqa: E402

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


class Drafts:
    """Queries, masks and outputs of drafted tokens over a Store."""

    def __init__(self, store, hq, drafts, most=None, mask=True, seed=0, words=None, form="plain"):
        g = torch.Generator(device="cuda").manual_seed(100 + seed)
        self.st, self.hq, self.drafts = store, hq, drafts
        self.most = most if most is not None else max(1, max(drafts))
        n = sum(drafts)
        self.q = torch.randn((n, hq, 128), generator=g, device="cuda").to(torch.bfloat16)
        if form == "heads":
            self.q = self.q.transpose(0, 1).contiguous().transpose(0, 1)
        s = [0]
        for d in drafts:
            s.append(s[-1] + d)
        self.starts = torch.tensor(s, dtype=torch.int32, device="cuda")
        words = words or (self.most + 31) // 32
        gc = torch.Generator().manual_seed(seed)
        self.mask = torch.cat([tree_bits(gc, d, words) for d in drafts]) if mask else None
        self.ws = T.alloc_workspace(T.tria_tree_workspace_size(store.stats, store.cache, self.most))
        self.out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, hq), 7.0, device="cuda")

    def run(self, layer=0, scale=SCALE, stream=None, lse=True):
        T.tria_tree_attention(self.st.stats, self.st.cache, layer, self.q, self.starts, self.most, scale, self.out,
                              self.ws, mask=self.mask, lse=self.lse if lse else None, stream=stream)

    def check(self, layer=0, scale=SCALE, seqs=None, heads=None, lens=None):
        st = self.st
        g = self.hq // st.hkv
        starts = self.starts.tolist()
        lens = lens if lens is not None else st.lens.tolist()
        for s in seqs if seqs is not None else range(len(self.drafts)):
            a, b, n = starts[s], starts[s + 1], lens[s]
            if a == b:
                continue
            sees = draft_sees(n, b - a, self.mask[a:b] if self.mask is not None else None)
            for h in heads if heads is not None else range(self.hq):
                k, v = (st.rows(x, layer, s, h // g, n + b - a) for x in (st.k, st.v))
                ref = attend(self.q[a:b, h], k, v, sees, scale)
                check(self.out[a:b, h], self.lse[a:b, h], ref, f"seq {s} head {h}")


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("mask", [True, False], ids=["tree", "chain"])
def test_matches_the_plain_form(hq, hkv, block, mask):
    lens, drafts = [0, 1, 126, 127, 128, 129, 700], [3, 1, 2, 9, 5, 0, 33]
    st = Store(T, 2, hq, hkv, lens, 768, block=block, seed=hq)
    try:
        st.idle = NAN
        st.spoil([n + d for n, d in zip(lens, drafts)])
        d = Drafts(st, hq, drafts, mask=mask, seed=1)
        d.run(layer=1)
        d.check(layer=1)
        assert T.tria_read_device_status(d.ws) == 0
    finally:
        st.free()


@pytest.mark.parametrize("block", [8, 16, 32, 64, 128])
def test_page_sizes_and_pages_that_end_inside_a_tile(block):
    lens, drafts = [1000, 5, 259], [7, 4, 1]
    st = Store(T, 1, 8, 2, lens, 1024, block=block, seed=block, idle=NAN)
    try:
        st.spoil([n + d for n, d in zip(lens, drafts)])
        d = Drafts(st, 8, drafts, seed=2)
        d.run()
        d.check()
    finally:
        st.free()


@pytest.mark.parametrize("n_draft", [1, 16, 17, 31, 32, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("mask", [True, False], ids=["tree", "chain"])
def test_draft_lengths(n_draft, mask):
    st = Store(T, 1, 16, 2, [333, 0], 700, seed=n_draft)
    try:
        d = Drafts(st, 16, [n_draft, n_draft], mask=mask, seed=3)
        d.run()
        d.check(heads=[0, 7, 8, 15])
    finally:
        st.free()


def test_long_context_split_over_many_blocks():
    st = Store(T, 1, 16, 2, [20011, 37], 20032, seed=4)
    try:
        d = Drafts(st, 16, [11, 3], seed=4)
        d.run()
        d.check()
    finally:
        st.free()


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("n_draft", [5, 40])
def test_many_key_blocks_and_several_units_for_each_processor(block, n_draft):
    # odd numbers of 64-key steps, units that begin and end inside a piece; again and again the same bits
    st = Store(T, 1, 32, 8, [20011, 6450, 13000], 20064, block=block, seed=15)
    try:
        d = Drafts(st, 32, [n_draft, 3, n_draft], seed=15)
        d.run()
        a, al = d.out.clone(), d.lse.clone()
        d.check(heads=[0, 13, 31])
        for _ in range(30):
            d.run()
        torch.cuda.synchronize()
        assert torch.equal(a, d.out) and torch.equal(al, d.lse)
        assert T.tria_read_device_status(d.ws) == 0
    finally:
        st.free()


def test_many_paged_sequences_of_different_lengths():
    lens = [(173 * i) % 1999 for i in range(40)]
    drafts = [(5 * i) % 13 for i in range(40)]
    st = Store(T, 1, 32, 8, lens, 2016, block=16, seed=5)
    try:
        d = Drafts(st, 32, drafts, seed=5)
        d.run()
        d.check(seqs=range(0, 40, 7), heads=[0, 3, 31])
    finally:
        st.free()


def test_rows_that_see_nothing():
    st = Store(T, 1, 8, 2, [0, 200, 0], 256, seed=6, idle=NAN)
    try:
        st.spoil([4, 204, 2])
        d = Drafts(st, 8, [4, 4, 2], seed=6)
        d.mask[1] = 0
        d.mask[5] = 0       # sees its committed rows alone
        d.mask[8:] = 0      # a sequence whose drafted tokens all see nothing
        d.run()
        d.check()
        assert bool((d.out[1] == 0).all()) and bool((d.lse[1] == -torch.inf).all())
    finally:
        st.free()


def test_any_mask_and_bits_behind_the_drafts():
    st = Store(T, 1, 8, 2, [90, 300], 400, seed=7, idle=NAN)
    try:
        st.spoil([90 + 40, 300 + 3])
        d = Drafts(st, 8, [40, 3], most=70, seed=7, words=4)
        g = torch.Generator(device="cuda").manual_seed(7)
        d.mask.copy_(torch.randint(-2 ** 31, 2 ** 31, d.mask.shape, generator=g, device="cuda"))
        d.run()
        d.check()
    finally:
        st.free()


@pytest.mark.parametrize("bad", [NAN, float("inf"), float("-inf")])
@pytest.mark.parametrize("block", [0, 16])
def test_what_a_token_does_not_see_does_not_reach_it(bad, block):
    st = Store(T, 1, 8, 2, [130, 0], 256, block=block, seed=8)
    try:
        d = Drafts(st, 8, [12, 12], seed=8)
        d.mask[:, 0] &= ~(1 << 5)
        d.mask[5, 0] = 1 << 5
        d.mask[12 + 5, 0] = 1 << 5       # node 5: seen by itself alone
        for s, n in enumerate([130, 0]):
            for x in (st.k, st.v):
                t = n + 5
                if block:
                    x[0, int(st.table[s, t // block]), t % block] = bad
                else:
                    x[0, s, :, t] = bad
        d.run()
        g, starts = 4, [0, 12]
        for s, n in enumerate([130, 0]):
            rows = [i for i in range(12) if i != 5]
            sees = draft_sees(n, 12, d.mask[starts[s]: starts[s] + 12])
            for h in range(8):
                k, v = (st.rows(x, 0, s, h // g, n + 12) for x in (st.k, st.v))
                k[n + 5], v[n + 5] = 0, 0
                at = [starts[s] + i for i in rows]
                ref = attend(d.q[at, h], k, v, sees[rows])
                check(d.out[at, h], d.lse[at, h], ref, (s, h))
        assert not bool(torch.isfinite(d.out[5].float()).all())
    finally:
        st.free()


def test_lengths_per_layer_and_strided_queries():
    lens = [300, 77]
    st = Store(T, 3, 8, 2, lens, 512, seed=9, layer_lens=True)
    try:
        st.layer_lens[0, 2], st.layer_lens[1, 2] = 41, 256
        d = Drafts(st, 8, [6, 2], seed=9, form="heads")
        d.run(layer=2)
        d.check(layer=2, lens=[41, 256])
        d.run(layer=1)
        d.check(layer=1, lens=lens)
    finally:
        st.free()


def test_block_ids_outside_the_pool_read_as_zero_rows():
    st = Store(T, 1, 8, 2, [100, 100], 128, block=16, seed=10)
    try:
        st.table[0, 2], st.table[1, 0] = -1, st.k.shape[1] + 5
        d = Drafts(st, 8, [3, 3], seed=10)
        d.run()
        d.check()
    finally:
        st.free()


def test_bad_sequences_are_flagged_and_left_alone():
    st = Store(T, 1, 8, 2, [100, 100, 100, 100], 128, seed=11)
    try:
        for change in ("len", "room", "draft", "starts"):
            d = Drafts(st, 8, [3, 3, 5, 3], most=5, seed=11)
            st.lens.copy_(torch.tensor([100, 100, 100, 100]))
            skipped = [1]
            if change == "len":
                st.lens[1] = -1
            elif change == "room":
                st.lens[1] = 126
            elif change == "draft":
                d.most, skipped = 4, [2]
            else:
                d.starts[4], skipped = 15, [3]
            d.run()
            assert T.tria_read_device_status(d.ws) == 1, change
            good = [s for s in range(4) if s not in skipped]
            d.check(seqs=good)
            a, b = (6, 11) if skipped == [2] else (3, 6) if skipped == [1] else (11, 14)
            assert bool((d.out[a:b] == 7.0).all()) and bool((d.lse[a:b] == 7.0).all()), change
    finally:
        st.free()


def test_one_drafted_token_is_a_decode_step():
    lens = [400, 31, 2000]
    st = Store(T, 1, 16, 2, lens, 2048, seed=12)
    try:
        d = Drafts(st, 16, [1, 1, 1], mask=False, seed=12)
        d.run()
        d.check()
        st.lens += 1
        out, lse = torch.empty((3, 16, 128), device="cuda"), torch.empty((3, 16), device="cuda")
        ws = T.alloc_workspace(T.tria_decode_workspace_size(st.stats, st.cache))
        T.tria_decode_attention(st.stats, st.cache, 0, d.q, SCALE, out, ws, lse=lse)
        assert float((out - d.out.float()).abs().max()) < 0.02 * float(out.abs().max())
        assert float((lse - d.lse).abs().max()) < 1e-4
    finally:
        st.free()


def test_equal_bits_on_another_stream_and_from_graphs():
    st = Store(T, 1, 32, 8, [3000, 50], 3100, seed=13)
    try:
        d = Drafts(st, 32, [9, 4], seed=13)
        e = Drafts(st, 32, [2, 70], seed=14, mask=False)
        need = max(d.ws.numel(), e.ws.numel())
        d.ws = e.ws = T.alloc_workspace(need)
        d.run()
        e.run()
        a, al, b = d.out.clone(), d.lse.clone(), e.out.clone()
        side = torch.cuda.Stream()
        d.out.fill_(1.0)
        side.wait_stream(torch.cuda.current_stream())
        d.run(stream=side)
        side.synchronize()
        assert torch.equal(a, d.out) and torch.equal(al, d.lse)
        graphs = []
        for x in (d, e):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                x.run()
            graphs.append(g)
        for _ in range(3):
            d.out.fill_(1.0)
            e.out.fill_(1.0)
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, d.out) and torch.equal(b, e.out)
        assert T.tria_read_device_status(d.ws) == 0
    finally:
        st.free()


def test_offsets_past_32_bits():
    # 16 sequences x 8 heads x 131300 rows x 128: the last rows lie past 2^31 elements
    lens = [0] * 15 + [131200]
    st = Store(T, 1, 16, 8, lens, 131300, seed=16)
    try:
        assert st.k.numel() > 2 ** 31
        d = Drafts(st, 16, [0] * 15 + [7], seed=16)
        d.run()
        d.check(heads=[0, 15])
        # the accepted rows of the last sequence, and a copy of it in the first
        want = [st.rows(x, 0, 15, 7, 131207)[131200 + torch.tensor([1, 4, 6], device="cuda")] for x in (st.k, st.v)]
        acc = torch.tensor([[0, 0, 0]] * 15 + [[1, 4, 6]], dtype=torch.int32, device="cuda")
        cnt = torch.tensor([0] * 15 + [3], dtype=torch.int32, device="cuda")
        ws = T.alloc_workspace(T.tria_commit_workspace_size(st.stats, st.cache))
        T.tria_tree_commit(st.stats, st.cache, acc, cnt, 0, 1, ws)
        wf = T.alloc_workspace(T.tria_fork_workspace_size(st.stats, st.cache))
        T.tria_fork_sequences(st.stats, st.cache, [15], [14], 0, 1, wf)
        for x, w in zip((st.k, st.v), want):
            assert torch.equal(st.rows(x, 0, 15, 7, 131203)[-3:], w)
            assert torch.equal(x[0, 14, :, :131203], x[0, 15, :, :131203])
        assert st.lens.tolist()[13:] == [0, 131203, 131203]
    finally:
        st.free()


def test_two_calls_at_once():
    st = Store(T, 1, 32, 8, [5000, 700], 5100, seed=17)
    try:
        d = Drafts(st, 32, [20, 3], seed=17)
        e = Drafts(st, 32, [3, 60], seed=18, mask=False)
        d.run()
        e.run()
        torch.cuda.synchronize()
        a, b = d.out.clone(), e.out.clone()
        d.out.fill_(1.0)
        e.out.fill_(1.0)
        one, two = torch.cuda.Stream(), torch.cuda.Stream()
        for s in (one, two):
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            d.run(stream=one)
            e.run(stream=two)
        torch.cuda.synchronize()
        assert torch.equal(a, d.out) and torch.equal(b, e.out)
        assert T.tria_read_device_status(d.ws) == 0 and T.tria_read_device_status(e.ws) == 0
    finally:
        st.free()
