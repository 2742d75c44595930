"""Cases of the decode operators around the paged K/V cache, for measuring them.

Five operators, each over a page pool that a block table maps:

  modified   decode attention whose scores are capped by a tanh, get a bias that
             grows with distance (one slope per head) or see a window only
  tree       decode attention for a tree of drafted tokens (an ancestor mask)
  weights    decode attention that also adds each cached token's softmax weight
             to a per-token sum
  evict      keep the tokens with the largest sums, in order, within a budget
  commit     move the accepted path of a drafted tree behind the context

``run`` computes them in plain torch operations in 32 bits, or, with ``own``
set, through the package's entry points; ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = dict(op=op, B=4, Hq=8, Hkv=2, page=16, lo=17, hi=256, q_len=1, layout="NHD", softcap=0.0,
             alibi=False, window=0, budget=0, sink=0, recent=0, in_place=True)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # a chat or two in an interactive session, capped scores: latency counts
        _case("modified", "cap_small", softcap=30.0),
        # a serving step of 64 sequences, capped scores
        _case("modified", "cap_serving", B=64, Hq=32, Hkv=8, lo=512, hi=4096, softcap=30.0),
        # local layer with a distance bias over long contexts, two tokens per step
        _case("modified", "window_alibi_long", B=8, Hq=32, Hkv=8, page=64, lo=32768, hi=131072,
              q_len=2, window=4096, alibi=True),
        # a small tree for a few interactive sequences
        _case("tree", "tree_small", q_len=8),
        # a serving step that verifies 16 drafted tokens per sequence
        _case("tree", "tree_16", B=64, Hq=32, Hkv=8, lo=512, hi=4096, q_len=16),
        # a large tree of 64 drafted tokens per sequence, capped scores
        _case("tree", "tree_64_cap", B=64, Hq=32, Hkv=8, lo=512, hi=4096, q_len=64, softcap=30.0),
        # a serving step that tracks which cached tokens are attended to
        _case("weights", "weights_serving", B=64, Hq=32, Hkv=8, lo=512, hi=4096),
        # the same over long contexts
        _case("weights", "weights_long", B=8, Hq=32, Hkv=8, page=64, lo=32768, hi=131072),
        # every sequence of a serving batch back to 2048 tokens, in its own pages
        _case("evict", "evict_serving", B=64, Hq=32, Hkv=8, lo=2049, hi=4096, budget=2048, sink=4,
              recent=256),
        # long prompts cut to 16384 tokens, into new pages (the old ones are shared)
        _case("evict", "evict_long", B=8, Hq=32, Hkv=8, page=64, lo=32768, hi=131072,
              budget=16384, sink=4, recent=1024, in_place=False),
        # the accepted path of a few small trees
        _case("commit", "commit_small", q_len=8),
        # and of a serving step with trees of 64 tokens
        _case("commit", "commit_64", B=64, Hq=32, Hkv=8, lo=512, hi=4096, q_len=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["modified", "modified", "tree", "tree", "weights", "evict", "commit"])
    Hq, Hkv = rng.choice([(8, 2), (32, 8), (64, 8), (32, 1), (8, 8), (16, 4), (12, 6), (5, 1),
                          (40, 8)])
    hi = _log_int(rng, 20, 60000)
    lo = rng.randint(max(1, hi // 8), hi)
    # at most the tokens x kv heads of a full serving step
    B = min(_log_int(rng, 1, 64), max(1, 64 * 4096 * 8 // (hi * Hkv)))
    c = dict(B=B, Hq=Hq, Hkv=Hkv, page=rng.choice([16, 32, 48, 64, 128]), lo=lo, hi=hi,
             layout=rng.choice(["NHD", "HND"]))
    if op in ("modified", "tree", "commit"):
        q_len = _log_int(rng, 2, 64) if op != "modified" else rng.choice([1, 1, 1, 2, 3, 5])
        c["q_len"] = q_len
        c["lo"], c["hi"] = max(c["lo"], q_len), max(c["hi"], q_len)
        # nor more products than the largest tree
        c["B"] = min(c["B"], max(1, 64 * 4096 * 32 * 64 // (c["hi"] * Hq * q_len)))
    if op in ("modified", "tree", "weights"):
        mods = rng.choice(["cap", "alibi", "window", "cap+window", "alibi+window"])
        if op != "modified" and rng.random() < 0.5:
            mods = ""
        if "cap" in mods:
            c["softcap"] = rng.choice([15.0, 30.0, 50.0])
        c["alibi"] = "alibi" in mods
        if "window" in mods:
            c["window"] = _log_int(rng, 16, 8192)
    if op == "evict":
        c["budget"] = max(8, int(hi * rng.uniform(0.1, 0.9)))
        c["sink"] = rng.randint(0, min(8, c["budget"] // 4))
        c["recent"] = rng.randint(0, c["budget"] // 2)
        c["in_place"] = rng.random() < 0.5
    return _case(op, **c)


# ------------------------------------------------------------------ structure
def _lens(c):
    """Lengths of the sequences: fixed by the case (the work depends on them)."""
    g = np.random.default_rng([c["B"], c["lo"], c["hi"]])
    lens = g.integers(c["lo"], c["hi"], size=c["B"], endpoint=True)
    lens[0] = c["hi"]
    return lens.astype(np.int64)


def _accepted(c):
    g = np.random.default_rng([c["B"], c["q_len"], 7])
    return g.integers(1, min(8, c["q_len"]), size=c["B"], endpoint=True)


def _drafted_trees(c, g):
    """Random trees: parents [B, q] (the parent's index, -1 at a root), every
    node after its parent; node 0 the root of all."""
    B, q = c["B"], c["q_len"]
    r = g.random((B, q))
    idx = np.arange(q)
    parents = np.floor(np.sqrt(r) * idx[None, :]).astype(np.int64)  # later nodes are likelier
    parents[:, 0] = -1
    seen = np.zeros((B, q, q), dtype=bool)
    for i in range(q):
        seen[:, i, i] = True
        if i:
            seen[:, i] |= seen[np.arange(B), parents[:, i]]
    return parents, seen


def _bits(seen):
    """bool [B, q, q] -> int32 words [B, q, ceil(q / 32)], bit j % 32 of word j / 32."""
    B, q, _ = seen.shape
    w = (q + 31) // 32
    pad = np.zeros((B, q, w * 32), dtype=np.uint64)
    pad[:, :, :q] = seen
    words = (pad.reshape(B, q, w, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def _slopes(c):
    return 2.0 ** (-8.0 * (torch.arange(c["Hq"], dtype=torch.float64) + 1) / c["Hq"])


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    g = np.random.default_rng([seed, 3])
    B, Hq, Hkv, P, q_len, D = c["B"], c["Hq"], c["Hkv"], c["page"], c["q_len"], 128
    lens = _lens(c)
    need = (lens + P - 1) // P
    used = int(need.sum())
    new = 0
    if c["op"] == "evict" and not c["in_place"]:
        new = int(((np.minimum(lens, c["budget"]) + P - 1) // P).sum())
    num_pages = int(math.ceil(1.25 * (used + new)))
    shape = (num_pages, P, Hkv, D) if c["layout"] == "NHD" else (num_pages, Hkv, P, D)

    def normal(shape, factor=1.0):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
        return x.mul_(factor) if factor != 1.0 else x

    perm = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)

    def table(counts, first):
        width = int(counts.max())
        t = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        cnt = torch.from_numpy(counts).to(DEV)
        start = first + torch.from_numpy(np.concatenate([[0], np.cumsum(counts)[:-1]])).to(DEV)
        col = torch.arange(width, device=DEV)
        ok = col[None, :] < cnt[:, None]
        idx = (start[:, None] + col[None, :]).clamp_(max=num_pages - 1)
        return torch.where(ok, perm[idx], t)

    s = dict(case=c, k=normal(shape), v=normal(shape), bt=table(need, 0),
             sl=torch.from_numpy(lens.astype(np.int32)).to(DEV), max_len=int(lens.max()),
             err=torch.zeros(1, dtype=torch.int32, device=DEV), scale=1.0 / math.sqrt(D))
    if c["op"] in ("modified", "tree", "weights"):
        s["q"] = normal((B, q_len, Hq, D), 2.0)
        s["out"] = torch.empty(B, q_len, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, q_len, Hq, dtype=torch.float32, device=DEV)
        s["slopes"] = _slopes(c).to(torch.float32).to(DEV) if c["alibi"] else None
    if c["op"] == "tree":
        _, seen = _drafted_trees(c, g)
        s["mask"] = torch.from_numpy(_bits(seen)).to(DEV)
    if c["op"] == "weights":
        s["weights"] = torch.rand(B, Hkv, s["max_len"], generator=gen, device=DEV)
    if c["op"] == "evict":
        w = torch.randn(B, Hkv, s["max_len"], generator=gen, device=DEV).mul_(2.0).exp_()
        # tokens nobody has attended to yet share the same sum
        w[torch.rand(w.shape, generator=gen, device=DEV) < 0.1] = 0.0
        s["weights"], s["weights_out"] = w, torch.zeros_like(w)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["kept"] = torch.zeros(B, Hkv, c["budget"], dtype=torch.int32, device=DEV)
        s["dst"] = None
        if not c["in_place"]:
            s["dst"] = table((np.minimum(lens, c["budget"]) + P - 1) // P, used)
    if c["op"] == "commit":
        parents, _ = _drafted_trees(c, g)
        acc = _accepted(c)
        path = np.full((B, q_len), -1, dtype=np.int32)
        for b in range(B):  # an ascending path from the root, as long as the tree allows
            node, n = 0, 0
            while n < acc[b]:
                path[b, n] = node
                n += 1
                kids = np.flatnonzero(parents[b] == node)
                if kids.size == 0:
                    break
                node = int(g.choice(kids))
            acc[b] = n
        s["path"] = torch.from_numpy(path).to(DEV)
        s["accepted"] = torch.from_numpy(acc.astype(np.int32)).to(DEV)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _nhd(pool, c):
    return pool if c["layout"] == "NHD" else pool.permute(0, 2, 1, 3)


def _rows(pool, bt, c):
    """The mapped rows of every sequence: [B, Hkv, T, D] in 32 bits (T = the table's reach)."""
    x = _nhd(pool, c)[bt.clamp(min=0).long()]  # [B, pages, P, Hkv, D]
    B, n, P, H, D = x.shape
    return x.reshape(B, n * P, H, D).permute(0, 2, 1, 3).float()


def _plain_attention(s):
    c = s["case"]
    B, q_len, Hq, D = s["q"].shape
    Hkv = c["Hkv"]
    g = Hq // Hkv
    k, v = _rows(s["k"], s["bt"], c), _rows(s["v"], s["bt"], c)
    T = k.shape[2]
    t = torch.arange(T, device=DEV)
    i = torch.arange(q_len, device=DEV)
    L = s["sl"].long()[:, None, None]
    ctx = L - q_len
    j = t[None, None, :] - ctx                                   # drafted index, [B, 1, T]
    if "mask" in s:
        shift = torch.arange(32, device=DEV)
        m = ((s["mask"][..., None] >> shift) & 1).bool().flatten(2)[:, :, :q_len]
        depth = (m.sum(2) - 1).clamp(min=0)                      # [B, q]
        m = torch.gather(m, 2, j.clamp(0, q_len - 1).expand(B, q_len, T))
        pos_t = torch.gather(depth, 1, j[:, 0].clamp(0, q_len - 1))[:, None, :] + ctx
        pos_t = torch.where(j < 0, t[None, None, :], pos_t)
        pos_i = depth[:, :, None] + ctx
        vis = (j < 0) | ((j < q_len) & m)
    else:
        pos_i = ctx + i[None, :, None]
        pos_t = t[None, None, :]
        vis = (pos_t <= pos_i) & (pos_t < L)
    dist = pos_i - pos_t                                         # [B, q, T]
    if c["window"]:
        vis = vis & (dist < c["window"])
    q = s["q"].float().view(B, q_len, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, q_len, g, T)
    del k
    if c["softcap"]:
        x = torch.tanh_(x.div_(c["softcap"])).mul_(c["softcap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, 1, g, 1) * dist[:, None, :, None, :].float()
    x = torch.where(vis[:, None, :, None, :], x, torch.full((), -math.inf, device=DEV))
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (x - top).exp_()
    den = p.sum(-1, keepdim=True)
    lse = (top + den.log()).squeeze(-1)
    p = p / den.clamp(min=1e-38)
    v = torch.where((t[None, :] < s["sl"][:, None])[:, None, :, None], v, torch.zeros((), device=DEV))
    out = torch.matmul(p.view(B, Hkv, -1, T), v).view(B, Hkv, q_len, g, D)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, q_len, Hq, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, q_len, Hq)
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    r = {"out": s["out"], "lse": s["lse"]}
    if "weights" in s:
        n = s["max_len"]
        inside = torch.arange(n, device=DEV)[None, None, :] < s["sl"][:, None, None]
        s["weights"].add_(torch.where(inside, p.sum((2, 3))[:, :, :n], torch.zeros((), device=DEV)))
        r["weights"] = s["weights"]
    return r


def _scatter(pool, c, page, slot, ok, rows):
    """rows [B, n, Hkv, D] into (page, slot) [B, Hkv, n] of the pool, where ok."""
    x = _nhd(pool, c)
    h = torch.arange(c["Hkv"], device=DEV)[None, :, None].expand_as(page)
    x[page[ok], slot[ok], h[ok]] = rows[ok]


def _gather(pool, c, page, slot):
    h = torch.arange(c["Hkv"], device=DEV)[None, :, None].expand_as(page)
    return _nhd(pool, c)[page, slot, h]


def _slots(bt, pos, P):
    """(page, slot) of positions [B, Hkv, n] through the block table."""
    B, H, n = pos.shape
    page = torch.gather(bt.long(), 1, (pos // P).reshape(B, -1)).view(B, H, n).clamp(min=0)
    return page, pos % P


def _plain_evict(s):
    c, w = s["case"], s["weights"]
    B, H, n = w.shape
    budget = c["budget"]
    L = s["sl"].long()[:, None, None]
    t = torch.arange(n, device=DEV)[None, None, :]
    always = (t < c["sink"]) | (t >= L - c["recent"])
    big = torch.full((), math.inf, device=DEV)
    key = torch.where(always, big, w)
    key = torch.where(t < L, key, -big)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :budget]
    count = L.clamp(max=budget)
    k = torch.arange(budget, device=DEV)[None, None, :]
    order = order if order.shape[2] == budget else torch.nn.functional.pad(
        order, (0, budget - order.shape[2]), value=n)
    kept = torch.where(k < count, order, n).sort(2).values  # unused places last
    ok = k < count
    src = torch.where(ok, kept, 0)
    P = c["page"]
    width = s["bt"].shape[1] * P
    page, slot = _slots(s["bt"], src.clamp(max=width - 1), P)
    dst_bt = s["bt"] if s["dst"] is None else s["dst"]
    dpage, dslot = _slots(dst_bt, k.expand(B, H, budget).clamp(max=dst_bt.shape[1] * P - 1), P)
    for pool in (s["k"], s["v"]):
        _scatter(pool, c, dpage, dslot, ok.expand(B, H, budget), _gather(pool, c, page, slot))
    m = min(budget, n)
    moved = torch.gather(w, 2, src[:, :, :m])
    s["weights_out"][:, :, :m] = torch.where(ok[:, :, :m], moved, s["weights_out"][:, :, :m])
    s["kept"].copy_(torch.where(ok, kept, -1))
    s["new_lens"].copy_(count[:, 0, 0])
    return {"k_pool": s["k"], "v_pool": s["v"], "weights": s["weights_out"], "kept": s["kept"],
            "new_lens": s["new_lens"]}


def _plain_commit(s):
    c = s["case"]
    B, q_len, H, P = c["B"], c["q_len"], c["Hkv"], c["page"]
    ctx = (s["sl"].long() - q_len)[:, None]
    j = torch.arange(q_len, device=DEV)[None, :]
    ok = j < s["accepted"].long()[:, None]
    src = ctx + s["path"].long().clamp(min=0)
    dst = ctx + j
    wide = lambda x: x[:, None, :].expand(B, H, q_len)  # noqa: E731
    page, slot = _slots(s["bt"], wide(src), P)
    dpage, dslot = _slots(s["bt"], wide(dst), P)
    for pool in (s["k"], s["v"]):
        _scatter(pool, c, dpage, dslot, wide(ok), _gather(pool, c, page, slot))
    s["new_lens"].copy_((ctx[:, 0] + s["accepted"]))
    return {"k_pool": s["k"], "v_pool": s["v"], "new_lens": s["new_lens"]}


# ----------------------------------------------------------- the package's own
def _own(s):
    import paged_decode_attention_gqa_gb300 as zl
    c = s["case"]
    if c["op"] in ("modified", "tree", "weights"):
        zl.decode_attn(s["q"], s["k"], s["v"], s["bt"], s["sl"], page_size=c["page"],
                       scale=s["scale"], out=s["out"], lse=s["lse"], err_flags=s["err"],
                       max_seq_len=s["max_len"], layout=c["layout"], softcap=c["softcap"],
                       alibi_slopes=s["slopes"], window=c["window"], tree_mask=s.get("mask"),
                       weights=s.get("weights"))
        r = {"out": s["out"], "lse": s["lse"]}
        if "weights" in s:
            r["weights"] = s["weights"]
        return r
    if c["op"] == "evict":
        zl.kv_evict(s["k"], s["v"], s["bt"], s["sl"], s["weights"], page_size=c["page"],
                    budget=c["budget"], sink=c["sink"], recent=c["recent"], layout=c["layout"],
                    new_lens=s["new_lens"], kept=s["kept"], weights_out=s["weights_out"],
                    dst_block_table=s["dst"], err_flags=s["err"])
        return {"k_pool": s["k"], "v_pool": s["v"], "weights": s["weights_out"],
                "kept": s["kept"], "new_lens": s["new_lens"]}
    zl.kv_commit(s["k"], s["v"], s["bt"], s["sl"], s["path"], s["accepted"], page_size=c["page"],
                 q_len=c["q_len"], layout=c["layout"], new_lens=s["new_lens"],
                 err_flags=s["err"])
    return {"k_pool": s["k"], "v_pool": s["v"], "new_lens": s["new_lens"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "evict":
        return _plain_evict(state)
    if op == "commit":
        return _plain_commit(state)
    return _plain_attention(state)


# --------------------------------------------------------------------- work
def work(case):
    c = dict(case)
    lens, D = _lens(c), 128
    B, Hq, Hkv, q_len, P = c["B"], c["Hq"], c["Hkv"], c["q_len"], c["page"]
    if c["op"] == "commit":
        moved = int(_accepted(c).sum()) * Hkv
        return {"bytes": moved * 2 * 2 * D * 2 + B * (q_len + 3) * 4, "flops": 0}
    if c["op"] == "evict":
        kept = int(np.minimum(lens, c["budget"]).sum()) * Hkv
        read_w = int(lens.sum()) * Hkv * 4
        return {"bytes": kept * (2 * 2 * D * 2 + 4 + 4) + read_w, "flops": 0}
    ctx = lens - q_len
    lo = np.maximum(ctx - c["window"] + 1, 0) if c["window"] else np.zeros_like(lens)
    seen = int((lens - lo).sum())
    nbytes = seen * Hkv * 2 * D * 2 + B * q_len * Hq * (2 * 2 * D + 4)
    nbytes += int(((lens - lo + P - 1) // P).sum()) * 4
    if c["op"] == "weights":
        nbytes += int(lens.sum()) * Hkv * 8
    return {"bytes": nbytes, "flops": 4 * seen * q_len * Hq * D}


# --------------------------------------------------------------------- exact
def _exact_attention(s):
    c = s["case"]
    B, q_len, Hq, D = s["q"].shape
    Hkv, P = c["Hkv"], c["page"]
    g = Hq // Hkv
    lens = s["sl"].tolist()
    out = torch.zeros(B, q_len, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, q_len, Hq), -math.inf, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if "weights" in s else None
    slopes = None if s["slopes"] is None else s["slopes"].double()
    words = s["mask"].cpu().numpy().view(np.uint32) if "mask" in s else None
    for b in range(B):
        L = lens[b]
        first = L - q_len
        see = torch.zeros(q_len, L, dtype=torch.bool)
        see[:, :first] = True
        at = torch.arange(L)                 # position of every cached token
        own_at = torch.arange(first, L)      # and of every query token
        for a in range(q_len):
            if words is None:
                see[a, first:first + a + 1] = True
            else:
                bits = [x for x in range(q_len) if (int(words[b, a, x // 32]) >> (x % 32)) & 1]
                see[a, [first + x for x in bits]] = True
                own_at[a] = first + max(len(bits) - 1, 0)
        at[first:] = own_at
        far = own_at[:, None] - at[None, :]
        if c["window"]:
            see &= far < c["window"]
        see, far = see.to(DEV), far.to(DEV)
        pages = s["bt"][b, torch.arange(L, device=DEV) // P].long()
        slots = torch.arange(L, device=DEV) % P
        for h in range(Hkv):
            if c["layout"] == "NHD":
                kk, vv = s["k"][pages, slots, h].double(), s["v"][pages, slots, h].double()
            else:
                kk, vv = s["k"][pages, h, slots].double(), s["v"][pages, h, slots].double()
            heads = range(h * g, (h + 1) * g)
            # a large group head by head, to hold fewer scores at once
            for a in heads if q_len * g * L > (1 << 26) else [slice(h * g, (h + 1) * g)]:
                qq = s["q"][b, :, a].double().reshape(q_len, -1, D)
                x = torch.einsum("qgd,td->qgt", qq, kk) * s["scale"]
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                if slopes is not None:
                    x = x - slopes[a].reshape(1, -1, 1) * far[:, None, :].double()
                x = x.masked_fill(~see[:, None, :], -math.inf)
                z = torch.logsumexp(x, 2)
                p = torch.where(torch.isinf(z)[..., None], 0.0, torch.exp(x - z[..., None]))
                out[b, :, a] = torch.einsum("qgt,td->qgd", p, vv).reshape(out[b, :, a].shape)
                lse[b, :, a] = z.reshape(lse[b, :, a].shape)
                if weights is not None:
                    weights[b, h, :L] += p.sum((0, 1))
    r = {"out": out, "lse": lse}
    if weights is not None:
        r["weights"] = weights
    return r


def _exact_moves(s, b, h, src, dst, dst_bt):
    """Copy rows src -> dst (positions) of kv head h of sequence b, all read first."""
    c, P = s["case"], s["case"]["page"]
    sp, ss = s["bt"][b, src // P].long(), src % P
    dp, ds = dst_bt[b, dst // P].long(), dst % P
    for pool in (s["k"], s["v"]):
        if c["layout"] == "NHD":
            pool[dp, ds, h] = pool[sp, ss, h].clone()
        else:
            pool[dp, h, ds] = pool[sp, h, ss].clone()


def _exact_evict(s):
    c = s["case"]
    lens, budget = s["sl"].tolist(), c["budget"]
    dst_bt = s["bt"] if s["dst"] is None else s["dst"]
    w64 = s["weights"].double().cpu().numpy()
    kept = np.full((c["B"], c["Hkv"], budget), -1, dtype=np.int32)
    wout = s["weights_out"].double()
    for b, L in enumerate(lens):
        for h in range(c["Hkv"]):
            keep = np.arange(L)
            if L > budget:
                mid = np.arange(c["sink"], L - c["recent"])
                best = mid[np.argsort(-w64[b, h, mid], kind="stable")[:budget - c["sink"] - c["recent"]]]
                keep = np.sort(np.concatenate([np.arange(c["sink"]), best, np.arange(L - c["recent"], L)]))
            kept[b, h, :len(keep)] = keep
            src = torch.from_numpy(keep).to(DEV)
            _exact_moves(s, b, h, src, torch.arange(len(keep), device=DEV), dst_bt)
            wout[b, h, :len(keep)] = s["weights"][b, h, src].double()
    new = torch.tensor([min(L, budget) for L in lens], dtype=torch.int32)
    return {"k_pool": s["k"], "v_pool": s["v"], "weights": wout, "kept": torch.from_numpy(kept),
            "new_lens": new}


def _exact_commit(s):
    c = s["case"]
    lens, path, acc = s["sl"].tolist(), s["path"].long(), s["accepted"].tolist()
    for b in range(c["B"]):
        first = lens[b] - c["q_len"]
        src = first + path[b, :acc[b]]
        for h in range(c["Hkv"]):
            _exact_moves(s, b, h, src, first + torch.arange(acc[b], device=DEV), s["bt"])
    new = torch.tensor([lens[b] - c["q_len"] + acc[b] for b in range(c["B"])], dtype=torch.int32)
    return {"k_pool": s["k"], "v_pool": s["v"], "new_lens": new}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    if case["op"] == "commit":
        return _exact_commit(s)
    return _exact_attention(s)
