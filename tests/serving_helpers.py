"""Plain 64-bit forms of the serving operators, and the tolerances that their
tests use.

Tolerance of an attention row over its keys, from the arithmetic:
  * a logit is a 128-term fp32 sum of exact bf16 products: within
    E = scale 2^-16 sum_d |q_d k_d| of the exact one;
  * so every softmax weight moves by at most 2 max_j E_j relative (doubled
    below for the second order), its exponential is evaluated within 2^-13,
    and it is rounded to bf16 (2^-8) before it multiplies a value;
  * the output is rounded to bf16 once (2^-8 of its size).
lse sums unrounded fp32 weights: 2 max_j E_j + 2e-5 (1 + |lse|).
"""
from __future__ import annotations

import torch

SCALE = 128 ** -0.5


def attend(q, k, v, allowed, scale=SCALE):
    """q [n, 128], k and v [m, 128] bf16, allowed [n, m] bool.  Returns fp64
    (out, lse, tol_out, tol_lse); a row that sees nothing has out 0, lse -inf.
    Rows of k and v that no row sees may hold anything."""
    seen = allowed.any(0)
    qd = q.double()
    kd = torch.where(seen[:, None], k.double(), 0.0)
    vd = torch.where(seen[:, None], v.double(), 0.0)
    z = torch.where(allowed, scale * (qd @ kd.T), -torch.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.where(allowed, torch.exp(z - lse[:, None]), 0.0)
    w = torch.where(lse[:, None] == -torch.inf, 0.0, w)
    out = w @ vd
    e = torch.where(allowed, scale * 2.0 ** -16 * (qd.abs() @ kd.abs().T), 0.0).amax(1, keepdim=True)
    size = w @ vd.abs()
    moved = size * (2.0 ** -8 + 2.0 ** -13 + 4 * e)
    tol_out = moved + 2.0 ** -8 * (out.abs() + moved) + 1e-30
    tol_lse = 2 * e[:, 0] + 2e-5 * (1 + torch.where(lse == -torch.inf, 0.0, lse).abs())
    return out, lse, tol_out, tol_lse


def check(out, lse, ref, where):
    r_out, r_lse, t_out, t_lse = ref
    d = (out.double() - r_out).abs()
    assert bool((d <= t_out).all()), (where, float((d / t_out).nan_to_num(1e9).max()))
    if lse is not None:
        none = r_lse == -torch.inf
        assert bool((lse[none] == -torch.inf).all()), where
        d = (lse.double() - r_lse).abs()[~none]
        assert bool((d <= t_lse[~none]).all()), (where, float((d / t_lse[~none]).nan_to_num(1e9).max()))


def causal(n, device="cuda"):
    i = torch.arange(n, device=device)
    return i[:, None] >= i[None, :]


def draft_sees(n_ctx, n_draft, bits=None, device="cuda"):
    """[n_draft, n_ctx + n_draft]: every committed row, and a chain's or the
    mask's (int32 words [n_draft, words]) drafted rows."""
    i = torch.arange(n_draft, device=device)
    if bits is None:
        d = i[:, None] >= i[None, :]
    else:
        d = ((bits.long()[:, i // 32] >> (i % 32)) & 1) == 1
    return torch.cat([torch.ones((n_draft, n_ctx), dtype=torch.bool, device=device), d], 1)


def tree_bits(gen, n_draft, words, device="cuda"):
    """Ancestor words of a random tree of n_draft nodes."""
    bits = []
    for i in range(n_draft):
        parent = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
        bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
    rows = [[(b >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for b in bits]
    return torch.tensor(rows, dtype=torch.int64).reshape(n_draft, words).to(torch.int32).to(device)


class Store:
    """A K/V cache of random rows (stacked layers) with its view; unused slots
    hold `idle`."""

    def __init__(self, T, layers, hq, hkv, lens, cap, block=0, seed=0, idle=0.0, positions=False,
                 layer_lens=False, spare=3, sigma=1.0):
        import numpy as np

        g = torch.Generator(device="cuda").manual_seed(seed)
        n_seq = len(lens)
        self.T, self.block, self.cap, self.hkv, self.layers = T, block, cap, hkv, layers
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.layer_lens = self.lens[:, None].repeat(1, layers).contiguous() if layer_lens else None
        self.positions = (torch.randint(0, 1 << 20, (n_seq, layers, hkv, cap), generator=g, device="cuda",
                                        dtype=torch.int32) if positions else None)
        if block:
            per = -(-cap // block)
            n_blocks = n_seq * per + spare
            self.table = torch.randperm(n_blocks, generator=g, device="cuda")[: n_seq * per].to(torch.int32)
            self.table = self.table.view(n_seq, per).contiguous()
            shape = (layers, n_blocks, block, hkv, 128)
        else:
            self.table = None
            shape = (layers, n_seq, hkv, cap, 128)
        self.k = (sigma * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)
        self.v = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        self.idle = idle
        self.make_view()
        ones = np.ones((layers, hq, 64), np.float32)
        self.stats = T.tria_load_stats(T.model_desc(layers, hq, hkv, T.PAIR_NEOX, 1e4), ones, ones, 2 * ones)

    def make_view(self):
        T, k = self.T, self.k
        lens = None if self.layer_lens is not None else self.lens
        kw = dict(positions=self.positions, layer_seq_lens=self.layer_lens, n_seq=self.lens.numel())
        if self.table is None:
            self.cache = T.Cache(T.LAYOUT_CONTIGUOUS, list(k.unbind(0)), list(self.v.unbind(0)), lens, None,
                                 self.cap, stride_seq=k.stride(1), stride_head=k.stride(2),
                                 stride_token=k.stride(3), **kw)
        else:
            self.cache = T.Cache(T.LAYOUT_PAGED, list(k.unbind(0)), list(self.v.unbind(0)), lens, None, self.cap,
                                 stride_head=k.stride(3), stride_token=k.stride(2), stride_block=k.stride(1),
                                 block_table=self.table, max_blocks_per_seq=self.table.shape[1],
                                 block_size=self.block, num_blocks=k.shape[1], **kw)

    def rows(self, x, layer, s, h, n):
        """Rows 0 .. n-1 of one unit (a copy)."""
        if self.table is None:
            return x[layer, s, h, :n].clone()
        b = self.table[s, : -(-n // self.block)].long()
        ok = (b >= 0) & (b < x.shape[1])
        got = x[layer, b.clamp(0, x.shape[1] - 1), :, h]
        return torch.where(ok[:, None, None], got, 0.0).reshape(-1, 128)[:n].clone()

    def spoil(self, used):
        """Every row that is no row 0 .. used[s]-1 of a sequence := idle (NaN)."""
        for x in (self.k, self.v):
            keep = torch.zeros(x.shape[1:-1], dtype=torch.bool, device="cuda")
            for s, n in enumerate(used):
                if self.table is None:
                    keep[s, :, :n] = True
                else:
                    t = torch.arange(n, device="cuda")
                    keep[self.table[s].long()[t // self.block], t % self.block] = True
            x[:, ~keep] = self.idle

    def free(self):
        self.stats.free()
