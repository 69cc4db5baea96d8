"""tria_tree_commit and tria_fork_sequences on the GPU: every byte of the cache
against a copy moved row by row, and the serving operators in one run."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import numpy as np  # noqa: E402

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import SCALE, Store, attend, causal, check, draft_sees, tree_bits  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


class Model:
    """Host copy of a Store, moved row by row."""

    def __init__(self, st):
        self.st = st
        self.k, self.v = (x.cpu().view(torch.int16).numpy().copy() for x in (st.k, st.v))
        self.pos = st.positions.cpu().numpy().copy() if st.positions is not None else None
        self.lens = (st.layer_lens if st.layer_lens is not None else st.lens).cpu().numpy().copy()
        self.table = st.table.cpu().numpy() if st.table is not None else None

    def len_of(self, s, layer):
        return int(self.lens[s, layer] if self.lens.ndim == 2 else self.lens[s])

    def at(self, s, t):
        """Index of slot t of sequence s behind the layer, and before the head."""
        if self.table is None:
            return s, slice(None), t
        return int(self.table[s, t // self.st.block]), t % self.st.block, slice(None)

    def move(self, layer, s_from, a, s_to, b):
        for x in (self.k, self.v):
            x[layer][self.at(s_to, b)] = x[layer][self.at(s_from, a)]

    def move_pos(self, layer, s_from, a, s_to, b):
        if self.pos is not None:
            self.pos[s_to, layer, :, b] = self.pos[s_from, layer, :, a]

    def same(self):
        st = self.st
        assert np.array_equal(st.k.cpu().view(torch.int16).numpy(), self.k)
        assert np.array_equal(st.v.cpu().view(torch.int16).numpy(), self.v)
        if self.pos is not None:
            assert np.array_equal(st.positions.cpu().numpy(), self.pos)
        got = st.layer_lens if st.layer_lens is not None else st.lens
        assert np.array_equal(got.cpu().numpy(), self.lens)


def commit(st, paths, layer0=0, layer1=None, width=None, ws=None, stream=None, counts=None):
    width = width or max(1, max(len(p) for p in paths))
    acc = torch.tensor([list(p) + [-5] * (width - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts or [len(p) for p in paths], dtype=torch.int32, device="cuda")
    ws = ws if ws is not None else T.alloc_workspace(T.tria_commit_workspace_size(st.stats, st.cache))
    T.tria_tree_commit(st.stats, st.cache, acc, cnt, layer0, st.layers if layer1 is None else layer1, ws, stream=stream)
    torch.cuda.synchronize()
    return ws


def model_commit(m, paths, layers, skip=(), grow=True):
    for s, path in enumerate(paths):
        if s in skip:
            continue
        for layer in layers:
            n = m.len_of(s, layer)
            for j, a in enumerate(path):
                m.move(layer, s, n + a, s, n + j)
                m.move_pos(layer, s, n + a, s, n + j)
            if m.lens.ndim == 2:
                m.lens[s, layer] += len(path)
        if m.lens.ndim == 1 and grow:
            m.lens[s] += len(path)


PATHS = [[], [0], [3], [0, 1, 2], [0, 2, 5, 6, 11], [1, 3]]


@pytest.mark.parametrize("block", [0, 8, 16, 128])
@pytest.mark.parametrize("hkv", [1, 2, 8])
@pytest.mark.parametrize("positions", [True, False])
def test_commit_moves_the_path_in_every_layer(block, hkv, positions):
    st = Store(T, 3, 8, hkv, [0, 7, 120, 127, 9, 243], 256, block=block, seed=1, positions=positions)
    try:
        m = Model(st)
        ws = commit(st, PATHS)
        model_commit(m, PATHS, range(3))
        m.same()
        assert T.tria_read_device_status(ws) == 0
        commit(st, [[1]] * 6, ws=ws)          # the counters are back at zero
        model_commit(m, [[1]] * 6, range(3))
        m.same()
    finally:
        st.free()


@pytest.mark.parametrize("block", [0, 16])
def test_commit_of_a_path_longer_than_one_chunk(block):
    path = sorted(set(range(0, 300)) - {0, 7, 100, 101, 250})
    st = Store(T, 2, 8, 8, [65, 3], 512, block=block, seed=2, positions=True)
    try:
        m = Model(st)
        commit(st, [path, path[:200]])
        model_commit(m, [path, path[:200]], range(2))
        m.same()
    finally:
        st.free()


@pytest.mark.parametrize("layer_lens", [True, False])
def test_commit_over_part_of_the_layers(layer_lens):
    st = Store(T, 4, 4, 2, [30, 40], 64, seed=3, layer_lens=layer_lens, positions=True)
    try:
        if layer_lens:
            st.layer_lens[1, 2] = 11
        m = Model(st)
        paths = [[1, 4], [0, 3, 4]]
        commit(st, paths, 0, 3)
        model_commit(m, paths, range(3), grow=False)
        m.same()
        commit(st, paths, 3, 4)
        model_commit(m, paths, [3])
        m.same()
    finally:
        st.free()


@pytest.mark.parametrize("path,count", [([2, 1], 2), ([1, 1], 2), ([-1, 0], 2), ([0, 64 - 20], 2), ([0, 1], 3), ([0, 1], -1)])
def test_commit_leaves_bad_paths_unchanged(path, count):
    st = Store(T, 2, 4, 2, [20, 20], 64, seed=4, positions=True)
    try:
        m = Model(st)
        ws = commit(st, [path, [3, 5]], counts=[count, 2])
        model_commit(m, [[], [3, 5]], range(2))
        m.same()
        assert T.tria_read_device_status(ws) == 1
        commit(st, [[0], [0]], ws=ws)
        model_commit(m, [[0], [0]], range(2))
        m.same()
        assert T.tria_read_device_status(ws) == 0
    finally:
        st.free()


def test_commit_with_bad_lengths_and_blocks():
    st = Store(T, 2, 4, 2, [20, 20, 20], 64, block=16, seed=5)
    try:
        st.lens[0] = 65
        m = Model(st)
        ws = commit(st, [[1], [1], [2]])
        model_commit(m, [[1], [1], [2]], range(2), skip=[0])
        m.same()
        assert T.tria_read_device_status(ws) == 1
        st.table[1, 1] = st.k.shape[1]         # slots 16 .. 31 of sequence 1
        m = Model(st)
        m.lens[1] += 1
        ws = commit(st, [[], [4], []], counts=[0, 1, 0])
        m.same()
        assert T.tria_read_device_status(ws) == 1
    finally:
        st.free()


def fork(st, src, dst, layer0=0, layer1=None, stream=None):
    ws = T.alloc_workspace(T.tria_fork_workspace_size(st.stats, st.cache))
    T.tria_fork_sequences(st.stats, st.cache, src, dst, layer0, st.layers if layer1 is None else layer1, ws,
                          stream=stream)
    torch.cuda.synchronize()
    return T.tria_read_device_status(ws)


def model_fork(m, src, dst, layers, grow=True):
    for a, b in zip(src, dst):
        for layer in layers:
            n = m.len_of(a, layer)
            for t in range(n):
                m.move(layer, a, t, b, t)
                m.move_pos(layer, a, t, b, t)
            if m.lens.ndim == 2:
                m.lens[b, layer] = n
        if m.lens.ndim == 1 and grow:
            m.lens[b] = m.lens[a]


@pytest.mark.parametrize("block", [0, 8, 32, 128])
@pytest.mark.parametrize("hkv", [1, 2, 8])
@pytest.mark.parametrize("positions", [True, False])
def test_fork_copies_rows_positions_and_length(block, hkv, positions):
    st = Store(T, 2, 8, hkv, [0, 63, 64, 65, 200, 9, 9, 9, 9, 9, 9], 256, block=block, seed=6, positions=positions)
    try:
        m = Model(st)
        src, dst = [4, 0, 4, 2, 4, 4, 4], [5, 6, 7, 8, 9, 10, 1]
        assert fork(st, src, dst) == 0
        model_fork(m, src, dst, range(2))
        m.same()
    finally:
        st.free()


def test_fork_shares_blocks_of_equal_table_entries():
    st = Store(T, 2, 8, 2, [100, 5, 5], 128, block=16, seed=7, positions=True)
    try:
        st.table[1, :6] = st.table[0, :6]      # whole blocks shared, slots 96 .. 99 copied
        st.table[2, :7] = st.table[0, :7]      # everything shared
        m = Model(st)
        assert fork(st, [0, 0], [1, 2]) == 0
        model_fork(m, [0, 0], [1, 2], range(2))
        m.same()
        shared = int(st.table[0, 6])
        assert int(st.table[1, 6]) != shared
        assert torch.equal(st.k[:, st.table[1, 6].long(), :4], st.k[:, shared, :4])
    finally:
        st.free()


@pytest.mark.parametrize("layer_lens", [True, False])
def test_fork_over_part_of_the_layers(layer_lens):
    st = Store(T, 3, 4, 2, [30, 40, 2], 64, seed=8, layer_lens=layer_lens, positions=True)
    try:
        if layer_lens:
            st.layer_lens[1, 1] = 11
        m = Model(st)
        assert fork(st, [1], [2], 1, 2) == 0
        model_fork(m, [1], [2], [1], grow=False)
        m.same()
        assert fork(st, [1], [2], 2, 3) == 0
        model_fork(m, [1], [2], [2])
        m.same()
    finally:
        st.free()


def test_fork_with_bad_lengths_and_blocks():
    st = Store(T, 1, 4, 2, [65, 40, 20, 20], 64, block=16, seed=9, positions=False)
    try:
        m = Model(st)
        assert fork(st, [0], [2]) == 1
        m.same()
        st.table[3, 1] = -1
        m = Model(st)
        assert fork(st, [1], [3]) == 1
        for t in list(range(16)) + list(range(32, 40)):
            m.move(0, 1, t, 3, t)
        m.lens[3] = 40
        m.same()
    finally:
        st.free()


def test_commit_and_fork_from_graphs():
    st = Store(T, 2, 8, 2, [50, 60, 1], 128, block=16, seed=10, positions=True)
    try:
        m = Model(st)
        acc = torch.tensor([[1, 3], [0, 2], [0, 0]], dtype=torch.int32, device="cuda")
        cnt = torch.tensor([2, 2, 0], dtype=torch.int32, device="cuda")
        ws = T.alloc_workspace(T.tria_commit_workspace_size(st.stats, st.cache))
        wf = T.alloc_workspace(T.tria_fork_workspace_size(st.stats, st.cache))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            T.tria_tree_commit(st.stats, st.cache, acc, cnt, 0, 2, ws)
            T.tria_fork_sequences(st.stats, st.cache, [1], [2], 0, 2, wf)
        for _ in range(3):
            g.replay()
            torch.cuda.synchronize()
            model_commit(m, [[1, 3], [0, 2], []], range(2))
            model_fork(m, [1], [2], range(2))
            m.same()
    finally:
        st.free()


@pytest.mark.parametrize("block", [0, 16])
def test_serving_run(block):
    """A prompt fills the cache, is forked, each copy is pruned by the pass,
    verifies a drafted tree, keeps a path and decodes: every step against the
    plain form on the rows that it should see."""
    L, hq, hkv, G, n0 = 2, 8, 2, 4, 700
    st = Store(T, L, hq, hkv, [n0, 0, 0], 1024, block=block, seed=11, positions=True)
    g = torch.Generator(device="cuda").manual_seed(12)
    try:
        q, k, v = (torch.randn((L, n0, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
        desc = T.model_desc(L, hq, hkv, T.PAIR_NEOX, 1e4)
        starts = torch.tensor([0, n0], dtype=torch.int32, device="cuda")
        wp = T.alloc_workspace(T.tria_prompt_workspace_size(desc, 1))
        out, lse = torch.empty((n0, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((n0, hq), device="cuda")
        for l in range(L):
            T.tria_prompt_attention(desc, q[l], k[l], v[l], starts, SCALE, out, wp, lse=lse)
            for h in range(hq):
                check(out[:, h], lse[:, h], attend(q[l, :, h], k[l, :, h // G], v[l, :, h // G], causal(n0)), (l, h))
            t = torch.arange(n0, device="cuda")
            for x, new in ((st.k, k[l]), (st.v, v[l])):
                if block:
                    x[l, st.table[0].long()[t // block], t % block] = new
                else:
                    x[l, 0, :, :n0] = new.transpose(0, 1)
        st.positions[0, :, :, :n0] = torch.arange(n0, dtype=torch.int32, device="cuda")
        assert fork(st, [0, 0], [1, 2]) == 0
        assert st.lens.tolist() == [n0] * 3

        # the pass: 256 rows of each copy stay
        qpos = torch.full((3,), n0 - 1, dtype=torch.int64, device="cuda")
        st.cache.view.query_pos = qpos.data_ptr()
        prm = T.params(256, 64, 4)
        wc = T.alloc_workspace(T.tria_workspace_size(st.stats, st.cache, prm))
        T.tria_read_device_status(wc)
        T.tria_compress_pass(st.stats, st.cache, prm, None, wc)
        assert st.lens.tolist() == [256] * 3
        for s in (1, 2):
            for l in range(L):
                assert torch.equal(st.rows(st.k, l, s, 1, 256), st.rows(st.k, l, 0, 1, 256))

        # drafted trees of 9, 1 and 4 tokens
        drafts, t0 = [9, 1, 4], [0, 9, 10]
        total = sum(drafts)
        gc = torch.Generator().manual_seed(13)
        mask = torch.cat([tree_bits(gc, d, 1) for d in drafts])
        ds = torch.tensor([0, 9, 10, 14], dtype=torch.int32, device="cuda")
        wt = T.alloc_workspace(T.tria_tree_workspace_size(st.stats, st.cache, 9))
        o = torch.empty((total, hq, 128), dtype=torch.bfloat16, device="cuda")
        ls = torch.empty((total, hq), device="cuda")
        for l in range(L):
            qt = torch.randn((total, hq, 128), generator=g, device="cuda").to(torch.bfloat16)
            T.tria_tree_attention(st.stats, st.cache, l, qt, ds, 9, SCALE, o, wt, mask=mask, lse=ls)
            for s, d in enumerate(drafts):
                a = t0[s]
                sees = draft_sees(256, d, mask[a: a + d])
                for h in range(hq):
                    kk, vv = (st.rows(x, l, s, h // G, 256 + d) for x in (st.k, st.v))
                    check(o[a: a + d, h], ls[a: a + d, h], attend(qt[a: a + d, h], kk, vv, sees), (l, s, h))

        m = Model(st)
        paths = [[0, 2, 5], [0], []]
        commit(st, paths)
        model_commit(m, paths, range(L))
        m.same()
        assert st.lens.tolist() == [259, 257, 256]

        qd = torch.randn((3, hq, 128), generator=g, device="cuda").to(torch.bfloat16)
        od, ld = torch.empty((3, hq, 128), device="cuda"), torch.empty((3, hq), device="cuda")
        wd = T.alloc_workspace(T.tria_decode_workspace_size(st.stats, st.cache))
        T.tria_decode_attention(st.stats, st.cache, 1, qd, SCALE, od, wd, lse=ld)
        for s, n in enumerate([259, 257, 256]):
            for h in range(hq):
                kk, vv = (st.rows(x, 1, s, h // G, n) for x in (st.k, st.v))
                ref = attend(qd[s: s + 1, h], kk, vv, torch.ones((1, n), dtype=torch.bool, device="cuda"))
                check(od[s: s + 1, h], ld[s: s + 1, h], ref, ("decode", s, h))
        for w in (wp, wt, wd):
            assert T.tria_read_device_status(w) == 0
    finally:
        st.free()
