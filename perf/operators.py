"""The serving operators next to the compression pass, as cases to measure:
attention over whole prompts, attention of drafted tokens over a cache, moving
the accepted drafted rows into place, and forking cached sequences.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the package's entry points.
"""
import math
import random

import torch

own = False

D = 128            # head dimension of the cache rows
SCALE = D ** -0.5
THETA = 1e4


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short question to a small model: one launch, latency counts
        dict(name="prompt_37", op="prompt", hq=8, hkv=2, n_seq=1, lo=37, hi=37, salt=1),
        # a serving batch of prompts of very different lengths, packed
        dict(name="prompt_ragged", op="prompt", hq=32, hkv=8, n_seq=24, lo=1, hi=2304, salt=2),
        # one prompt of the 36-layer 32q/8kv shape (8448 tokens)
        dict(name="prompt_8448", op="prompt", hq=32, hkv=8, n_seq=1, lo=8448, hi=8448, salt=3),
        # half of the 64q/8kv shape's 32K context in one prompt
        dict(name="prompt_16384", op="prompt", hq=64, hkv=8, n_seq=1, lo=16384, hi=16384, salt=4),
        # a handful of drafted tokens of the tiny shape: latency
        dict(name="tree_5", op="tree", hq=8, hkv=2, n_seq=1, lo=2304, hi=2304, t_lo=5, t_hi=5, chain=False,
             block=0, salt=5),
        # 64 paged sequences after compression to 2048 rows, trees of different sizes
        dict(name="tree_pruned_batch", op="tree", hq=32, hkv=8, n_seq=64, lo=2048, hi=2175, t_lo=1, t_hi=16,
             chain=False, block=16, salt=6),
        # a 16-node tree over the full 32K cache of the 64q/8kv shape
        dict(name="tree_32768", op="tree", hq=64, hkv=8, n_seq=1, lo=32768, hi=32768, t_lo=16, t_hi=16, chain=False,
             block=0, salt=7),
        # a chain of 64 drafted tokens over the 131K cache
        dict(name="chain_131072", op="tree", hq=64, hkv=8, n_seq=1, lo=131072, hi=131072, t_lo=64, t_hi=64, chain=True,
             block=0, salt=8),
        # the accepted path of one sequence, every layer of the 36-layer shape
        dict(name="commit_one", op="commit", layers=36, hkv=8, n_seq=1, lo=2048, hi=2048, draft=16, a_lo=4, a_hi=4,
             block=0, salt=9),
        # the accepted paths of 64 paged sequences, 32 layers
        dict(name="commit_batch", op="commit", layers=32, hkv=8, n_seq=64, lo=512, hi=1024, draft=32, a_lo=0, a_hi=12,
             block=16, salt=10),
        # three samples share a prompt's whole blocks; only the block being filled is copied
        dict(name="fork_shared", op="fork", layers=32, hkv=8, parents=1, kids=3, lo=2309, hi=2309, shared=True,
             block=16, salt=11),
        # private copies of two sequences for two children each (a pass that compacts in place comes next)
        dict(name="fork_private", op="fork", layers=32, hkv=8, parents=2, kids=2, lo=2000, hi=4097, shared=False,
             block=16, salt=12),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "commit", "fork"])
    salt = rng.randrange(1, 1 << 30)
    block = rng.choice([0, 8, 16, 32, 64, 128])
    if op == "prompt":
        hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 16])
        n_seq = _between(rng, 1, 64)
        hi = _between(rng, 1, min(12000, math.isqrt(15_000_000_000 // (hkv * g * n_seq))))
        return dict(op=op, hq=hkv * g, hkv=hkv, n_seq=n_seq, lo=_between(rng, 1, hi), hi=hi, salt=salt)
    if op == "tree":
        hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 16])
        n_seq = _between(rng, 1, 64)
        hi = _between(rng, 1, 65536 // n_seq)
        t_hi = _between(rng, 1, 48)
        return dict(op=op, hq=hkv * g, hkv=hkv, n_seq=n_seq, lo=_between(rng, 1, hi), hi=hi, t_lo=_between(rng, 1, t_hi),
                    t_hi=t_hi, chain=rng.random() < 0.3, block=block, salt=salt)
    if op == "commit":
        n_seq, draft = _between(rng, 1, 48), _between(rng, 2, 64)
        hi = _between(rng, 1, 16384 // n_seq)
        return dict(op=op, layers=_between(rng, 1, 36), hkv=rng.choice([1, 2, 4, 8]), n_seq=n_seq, lo=_between(rng, 1, hi),
                    hi=hi, draft=draft, a_lo=0, a_hi=_between(rng, 1, draft), block=block, salt=salt)
    hi = _between(rng, 1, 3000)
    return dict(op=op, layers=_between(rng, 1, 36), hkv=rng.choice([1, 2, 4, 8]), parents=_between(rng, 1, 3),
                kids=_between(rng, 1, 3), lo=_between(rng, 1, hi), hi=hi, shared=rng.random() < 0.5, block=block, salt=salt)


def _lengths(case, n, lo, hi, salt):
    rng = random.Random(1000003 * case["salt"] + salt)
    return [_between(rng, lo, hi) for _ in range(n)]


def _sizes(case):
    """Host-side sizes of a case: what the scheduler of a serving program knows."""
    if case["op"] == "prompt":
        return _lengths(case, case["n_seq"], case["lo"], case["hi"], 1), None
    if case["op"] == "tree":
        return (_lengths(case, case["n_seq"], case["lo"], case["hi"], 1),
                _lengths(case, case["n_seq"], case["t_lo"], case["t_hi"], 2))
    if case["op"] == "commit":
        rng = random.Random(1000003 * case["salt"] + 2)
        return (_lengths(case, case["n_seq"], case["lo"], case["hi"], 1),
                [rng.randint(case["a_lo"], case["a_hi"]) for _ in range(case["n_seq"])])
    return _lengths(case, case["parents"], case["lo"], case["hi"], 1), None


def work(case):
    """Bytes read once and written once, and the attention's multiply-adds."""
    lens, more = _sizes(case)
    if case["op"] == "prompt":
        t, hq, hkv = sum(lens), case["hq"], case["hkv"]
        return {"bytes": t * (hq * D * 4 + hkv * D * 4 + hq * 4), "flops": 4 * D * hq * sum(n * (n + 1) // 2 for n in lens)}
    if case["op"] == "tree":
        hq, hkv, rows, t = case["hq"], case["hkv"], sum(lens) + sum(more), sum(more)
        return {"bytes": rows * hkv * D * 4 + t * hq * (D * 4 + 4),
                "flops": 4 * D * hq * sum(b * (n + b // 2) for n, b in zip(lens, more))}
    units = case["layers"] * case["hkv"]
    if case["op"] == "commit":
        return {"bytes": units * sum(more) * (2 * D * 2 + 4) * 2 + 4 * sum(more) + 12 * len(lens), "flops": 0}
    bs = case["block"]
    rows = [n % bs if case["shared"] and bs else n for n in lens]
    return {"bytes": units * sum(rows) * (2 * D * 2) * (1 + case["kids"]) + units * sum(lens) * 4 * (1 + case["kids"]) + 64,
            "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rotated(x, pos):
    """x [..., n, heads, D] rotated by RoPE (half split) at pos [..., n]."""
    om = THETA ** (-2.0 * torch.arange(D // 2, device=x.device, dtype=torch.float64) / D)
    ang = torch.remainder(pos.double()[..., None] * om, 2 * math.pi).float()
    c, s = torch.cos(ang)[..., None, :], torch.sin(ang)[..., None, :]
    a, b = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1)


def _keys(gen, pos, heads, sigma):
    """Rows of concentrated heads: a center for each head, and noise for each token."""
    center = sigma * torch.randn((heads, D), generator=gen, device="cuda")
    x = center + 0.5 * torch.randn((*pos.shape, heads, D), generator=gen, device="cuda")
    return _rotated(x, pos).to(torch.bfloat16)


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def _tree_masks(case, drafts):
    """Ancestor bits of every drafted token, int32 words: node i of a random tree
    sees itself and its parents up to the root."""
    rng = random.Random(1000003 * case["salt"] + 3)
    words = (max(drafts) + 31) // 32
    rows = []
    for t in drafts:
        bits = []
        for i in range(t):
            parent = rng.randint(max(-1, i - 4), i - 1)
            bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
        rows += [[(b >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for b in bits]
    return torch.tensor(rows, dtype=torch.int64, device="cuda").to(torch.int32)


def _table(gen, n_seq, cap, block):
    """Block table of n_seq sequences with room for cap rows each, in random order."""
    per = -(-cap // block)
    return torch.randperm(n_seq * per, generator=gen, device="cuda").to(torch.int32).view(n_seq, per)


def _cache_of(T, case, st):
    """The package's view of the cache tensors of a state."""
    k, v, table = st["k"], st["v"], st["table"]
    if table is None:
        _, _, _, cap, _ = k.shape
        return T.Cache(T.LAYOUT_CONTIGUOUS, list(k.unbind(0)), list(v.unbind(0)), st["lens"], None, cap,
                       stride_seq=k.stride(1), stride_head=k.stride(2), stride_token=k.stride(3), positions=st.get("positions"))
    return T.Cache(T.LAYOUT_PAGED, list(k.unbind(0)), list(v.unbind(0)), st["lens"], None, st["cap"],
                   stride_head=k.stride(3), stride_token=k.stride(2), stride_block=k.stride(1), block_table=table,
                   max_blocks_per_seq=table.shape[1], block_size=k.shape[2], num_blocks=k.shape[1],
                   positions=st.get("positions"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + 7)
    lens, more = _sizes(case)
    st = {"op": case["op"], "case": case}
    if case["op"] == "prompt":
        hq, hkv, total = case["hq"], case["hkv"], sum(lens)
        pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
        # the projections of all heads lie side by side in one tensor, as a model's fused layer writes them
        qkv = torch.empty((total, hq + 2 * hkv, D), dtype=torch.bfloat16, device="cuda")
        qkv[:, :hq] = _keys(gen, pos, hq, 1.0)
        qkv[:, hq: hq + hkv] = _keys(gen, pos, hkv, 2.0)
        qkv[:, hq + hkv:] = torch.randn((total, hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
        st.update(q=qkv[:, :hq], k=qkv[:, hq: hq + hkv], v=qkv[:, hq + hkv:], starts=_starts(lens), longest=max(lens))
        st["out"] = torch.empty((total, hq, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((total, hq), device="cuda")
        if own:
            import key_retention_scoring_b200 as T
            st["T"], st["desc"] = T, T.model_desc(1, hq, hkv, T.PAIR_NEOX, THETA)
            st["ws"] = T.alloc_workspace(T.tria_prompt_workspace_size(st["desc"], case["n_seq"]))
        return st

    hkv, block = case["hkv"], case["block"]
    layers = case.get("layers", 1)
    n_seq = case["parents"] * (1 + case["kids"]) if case["op"] == "fork" else case["n_seq"]
    extra = {"tree": max(more) if case["op"] == "tree" else 0, "commit": case.get("draft", 0), "fork": 0}[case["op"]]
    cap = max(lens) + extra
    st["cap"], st["table"] = cap, _table(gen, n_seq, cap, block) if block else None
    if case["op"] == "fork":
        # parents first, then the children of each
        lens_now = lens + [0] * (n_seq - len(lens))
        src = [p for p in range(case["parents"]) for _ in range(case["kids"])]
        dst = list(range(case["parents"], n_seq))
        if block and case["shared"]:
            for a, b in zip(src, dst):
                st["table"][b, : lens[a] // block] = st["table"][a, : lens[a] // block]
        st["src"], st["dst"] = src, dst  # the scheduler's lists
    else:
        lens_now = lens
    st["lens"] = torch.tensor(lens_now, dtype=torch.int32, device="cuda")
    shape = (layers, n_seq, hkv, cap, D) if not block else (layers, st["table"].numel(), block, hkv, D)
    if case["op"] == "tree":
        pos = torch.arange(cap, device="cuda").expand(n_seq, cap)
        rows = _keys(gen, pos, hkv, 2.0)                       # [n_seq, cap, hkv, D]
        if block:
            k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            slot = torch.arange(cap, device="cuda")
            k[0, st["table"].long()[:, slot // block], (slot % block).expand(n_seq, cap)] = rows
        else:
            k = rows.permute(0, 2, 1, 3).contiguous()[None]
        st["k"], st["v"] = k, torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
        hq = case["hq"]
        tpos = torch.cat([n + torch.arange(t, device="cuda") for n, t in zip(lens, more)])
        st["q"] = _keys(gen, tpos, hq, 1.0)
        st["starts"], st["most"], st["longest"] = _starts(more), max(more), cap
        st["mask"] = None if case["chain"] else _tree_masks(case, more)
        st["out"] = torch.empty((sum(more), hq, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((sum(more), hq), device="cuda")
    else:
        st["k"], st["v"] = (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        st["positions"] = torch.randint(0, 1 << 20, (n_seq, layers, hkv, cap), generator=gen, device="cuda", dtype=torch.int32)
        hq = hkv
    if case["op"] == "commit":
        rng = random.Random(1000003 * case["salt"] + 4 + seed)
        acc = [sorted(rng.sample(range(case["draft"]), a)) for a in more]
        width = max(1, max(more))
        st["accepted"] = torch.tensor([a + [-1] * (width - len(a)) for a in acc], dtype=torch.int32, device="cuda")
        st["n_accepted"] = torch.tensor(more, dtype=torch.int32, device="cuda")
        st["lens0"] = st["lens"].clone()
    if own:
        import numpy as np
        import key_retention_scoring_b200 as T
        a = np.ones((layers, hq, D // 2), np.float32)
        st["T"], st["layers"] = T, layers
        st["stats"] = T.tria_load_stats(T.model_desc(layers, hq, hkv, T.PAIR_NEOX, THETA), a, a, 2 * a)
        st["cache"] = _cache_of(T, case, st)
        if case["op"] == "tree":
            n = T.tria_tree_workspace_size(st["stats"], st["cache"], st["most"])
        elif case["op"] == "commit":
            n = T.tria_commit_workspace_size(st["stats"], st["cache"])
        else:
            n = T.tria_fork_workspace_size(st["stats"], st["cache"])
        st["ws"] = T.alloc_workspace(n)
    return st


# ---------------------------------------------------------------------------
# plain forms, 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _softmax_rows(sc, allowed):
    """Weights, their sums and the log of the sums of exp over the last axis."""
    sc = sc.masked_fill_(~allowed, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    tot = p.sum(-1, keepdim=True)
    return p, tot, (m + torch.log(tot))[..., 0]


def _plain_prompt(st):
    q, k, v, starts, longest = st["q"], st["k"], st["v"], st["starts"].long(), st["longest"]
    hkv, g = k.shape[1], q.shape[1] // k.shape[1]
    at = torch.arange(longest, device=q.device)
    valid = at < (starts[1:] - starts[:-1])[:, None]                 # [n_seq, longest]
    idx = torch.where(valid, starts[:-1, None] + at, 0)
    allowed = (at[:, None] >= at)[None, None] & valid[:, None, None, :]
    out, lse = st["out"], st["lse"]
    # one KV head at a time: the scores of all heads of a long prompt do not fit the card
    for h in range(hkv):
        qh = q[:, h * g: (h + 1) * g].float()[idx].transpose(1, 2)   # [n_seq, g, longest, D]
        kh, vh = k[:, h].float()[idx][:, None], v[:, h].float()[idx][:, None]
        p, tot, ls = _softmax_rows((qh @ kh.transpose(-1, -2)).mul_(SCALE), allowed)
        o = (p @ vh) / tot
        out[:, h * g: (h + 1) * g] = o.transpose(1, 2)[valid].to(out.dtype)
        lse[:, h * g: (h + 1) * g] = ls.transpose(1, 2)[valid]
    return {"out": out, "lse": lse}


def _rows_of(x, table, slots):
    """Rows [n_seq, n, hkv, D] of the layer x at slots [n_seq, n]."""
    s = torch.arange(slots.shape[0], device=x.device)[:, None]
    if table is None:
        return x[s, :, slots]
    bs = x.shape[1]
    return x[table.long()[s, slots // bs], slots % bs]


def _plain_tree(st):
    q, starts, lens, most = st["q"], st["starts"].long(), st["lens"].long(), st["most"]
    n_seq, cap = lens.numel(), st["longest"]
    slots = torch.arange(cap, device=q.device).expand(n_seq, cap)
    k = _rows_of(st["k"][0], st["table"], slots).float().permute(0, 2, 1, 3)   # [n_seq, hkv, cap, D]
    v = _rows_of(st["v"][0], st["table"], slots).float().permute(0, 2, 1, 3)
    hkv = k.shape[1]
    g = q.shape[1] // hkv
    node = torch.arange(most, device=q.device)
    valid = node < (starts[1:] - starts[:-1])[:, None]                         # [n_seq, most]
    idx = torch.where(valid, starts[:-1, None] + node, 0)
    qs = q.float()[idx].view(n_seq, most, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(n_seq, hkv, most * g, D)
    rel = slots - lens[:, None]                                                # drafted node in a slot
    if st["mask"] is None:
        sees = rel[:, None, :] <= node[:, None]
    else:
        bits = (st["mask"].long()[:, :, None] >> torch.arange(32, device=q.device)) & 1
        bits = bits.reshape(bits.shape[0], -1)[idx]                            # [n_seq, most, 32 words]
        at = rel.clamp(0, bits.shape[-1] - 1)[:, None, :].expand(n_seq, most, cap)
        sees = (rel < 0)[:, None, :] | ((rel < bits.shape[-1])[:, None, :] & (bits.gather(2, at) == 1))
    allowed = sees[:, None, :, None, :].expand(n_seq, 1, most, g, cap).reshape(n_seq, 1, most * g, cap)
    p, tot, ls = _softmax_rows((qs @ k.transpose(-1, -2)).mul_(SCALE), allowed)
    o = ((p @ v) / tot).view(n_seq, hkv, most, g, D).permute(0, 2, 1, 3, 4).reshape(n_seq, most, hkv * g, D)
    ls = ls.view(n_seq, hkv, most, g).permute(0, 2, 1, 3).reshape(n_seq, most, hkv * g)
    st["out"].copy_(o[valid])
    st["lse"].copy_(ls[valid])
    return {"out": st["out"], "lse": st["lse"]}


def _plain_commit(st):
    lens, acc, cnt, table = st["lens"].long(), st["accepted"].long(), st["n_accepted"].long(), st["table"]
    j = torch.arange(acc.shape[1], device=lens.device)
    s = torch.arange(lens.numel(), device=lens.device)[:, None].expand_as(acc)
    dst = lens[:, None] + j
    src = torch.where(j < cnt[:, None], lens[:, None] + acc, dst)  # past the path: a row stays
    for x in (st["k"], st["v"]):
        if table is None:
            x[:, s, :, dst] = x[:, s, :, src]
        else:
            bs = x.shape[2]
            x[:, table.long()[s, dst // bs], dst % bs] = x[:, table.long()[s, src // bs], src % bs]
    pos = st["positions"]
    pos[s, :, :, dst] = pos[s, :, :, src]
    st["lens"] += st["n_accepted"]
    return {"k": st["k"], "v": st["v"], "positions": pos, "lens": st["lens"]}


def _plain_fork(st):
    lens, table = st["lens"], st["table"]
    src, dst = torch.tensor(st["src"], device=lens.device), torch.tensor(st["dst"], device=lens.device)
    at = torch.arange(st["cap"], device=src.device)
    moves = at < lens.long()[src][:, None]                 # [children, cap]
    if table is not None:
        blk = at // st["k"].shape[2]
        moves &= table[src][:, blk] != table[dst][:, blk]  # equal entries: the block is shared
    pos = st["positions"]
    pos[dst] = torch.where((at < lens.long()[src][:, None])[:, None, None, :], pos[src], pos[dst])
    i, slot = moves.nonzero(as_tuple=True)
    for x in (st["k"], st["v"]):
        if table is None:
            x[:, dst[i], :, slot] = x[:, src[i], :, slot]
        else:
            bs = x.shape[2]
            b, off = slot // bs, slot % bs
            x[:, table.long()[dst[i], b], off] = x[:, table.long()[src[i], b], off]
    lens[dst] = lens[src]
    return {"k": st["k"], "v": st["v"], "positions": pos, "lens": lens}


def run(st):
    if st["op"] == "commit":
        st["lens"].copy_(st["lens0"])  # the lengths that the step began with
    if not own:
        return {"prompt": _plain_prompt, "tree": _plain_tree, "commit": _plain_commit, "fork": _plain_fork}[st["op"]](st)
    T = st["T"]
    if st["op"] == "prompt":
        T.tria_prompt_attention(st["desc"], st["q"], st["k"], st["v"], st["starts"], SCALE, st["out"], st["ws"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if st["op"] == "tree":
        T.tria_tree_attention(st["stats"], st["cache"], 0, st["q"], st["starts"], st["most"], SCALE, st["out"], st["ws"],
                              mask=st["mask"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if st["op"] == "commit":
        T.tria_tree_commit(st["stats"], st["cache"], st["accepted"], st["n_accepted"], 0, st["layers"], st["ws"])
    else:
        T.tria_fork_sequences(st["stats"], st["cache"], st["src"], st["dst"], 0, st["layers"], st["ws"])
    return {"k": st["k"], "v": st["v"], "positions": st["positions"], "lens": st["lens"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence after another
# ---------------------------------------------------------------------------
def _attend(q, k, v, allowed):
    """q [n, D], k and v [m, D], allowed [n, m] or None: out [n, D], lse [n]."""
    z = torch.mm(q, k.t()) * SCALE
    if allowed is not None:
        z = torch.where(allowed, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, 1)
    return torch.mm(torch.exp(z - lse[:, None]), v), lse


def _seq_rows(x, table, s, n):
    """Rows 0 .. n-1 of sequence s of a stacked cache x, [layers, hkv, n, D] (a copy)."""
    if table is None:
        return x[:, s, :, :n].clone()
    bs = x.shape[2]
    blocks = table[s, : -(-n // bs)].long()
    return x[:, blocks].flatten(1, 2)[:, :n].transpose(1, 2).contiguous()


def _put_row(x, table, s, t, rows):
    """Row t of sequence s := rows [layers, hkv, D]."""
    if table is None:
        x[:, s, :, t] = rows
    else:
        x[:, int(table[s, t // x.shape[2]]), t % x.shape[2]] = rows


def exact(case, seed):
    st = prepare(case, seed)
    lens, more = _sizes(case)
    if case["op"] in ("prompt", "tree"):
        q = st["q"].double()
        out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        g = q.shape[1] // case["hkv"]
        first = 0
        for s, n in enumerate(lens):
            t = n if case["op"] == "prompt" else more[s]
            for h in range(case["hkv"]):
                if case["op"] == "prompt":
                    k, v = (x[first: first + n, h].double() for x in (st["k"], st["v"]))
                else:
                    k, v = (_seq_rows(x[:, :, h: h + 1] if st["table"] is None else x[:, :, :, h: h + 1], st["table"], s,
                                      n + t)[0, 0].double() for x in (st["k"], st["v"]))
                for hh in range(h * g, (h + 1) * g):
                    for a in range(0, t, 4096):
                        b = min(t, a + 4096)
                        end = b if case["op"] == "prompt" else n + t
                        i, j = torch.arange(a, b, device="cuda")[:, None], torch.arange(end, device="cuda")
                        if case["op"] == "prompt":
                            allowed = j <= i
                        elif case["chain"]:
                            allowed = j - n <= i
                        else:
                            rows = st["mask"][first + a: first + b].long()
                            d = torch.clamp(j - n, min=0)
                            allowed = (j < n) | (((rows[:, d // 32] >> (d % 32)) & 1) != 0)
                        out[first + a: first + b, hh], lse[first + a: first + b, hh] = _attend(
                            q[first + a: first + b, hh], k[:end], v[:end], allowed)
            first += t
        return {"out": out, "lse": lse}
    k, v, table = st["k"].double(), st["v"].double(), st["table"]
    if case["op"] == "commit":
        for s, n in enumerate(lens):
            path = st["accepted"][s, : more[s]].tolist()
            for x in (k, v):
                rows = _seq_rows(x, table, s, n + case["draft"])
                for j, node in enumerate(path):
                    _put_row(x, table, s, n + j, rows[:, :, n + node])
    else:
        for a, b in zip(st["src"], st["dst"]):
            for x in (k, v):
                n = lens[a]
                if table is None:
                    x[:, b, :, :n] = x[:, a, :, :n]
                else:
                    rows = _seq_rows(x, table, a, n)                   # [layers, hkv, n, D]
                    for c in range(-(-n // case["block"])):
                        part = rows[:, :, c * case["block"]: (c + 1) * case["block"]]
                        x[:, int(table[b, c]), : part.shape[2]] = part.transpose(1, 2)
    return {"k": k, "v": v, "positions": None, "lens": None}
