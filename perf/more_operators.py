"""Cases of the decode step over a K/V cache held in 4 bits, for measuring them.

Four operators, each over heads of 128 elements:

  attn       decode attention over a paged cache of 4-bit rows
  cache      new tokens' K and V rows quantised into the pages as they are
             written, then the sequences' tokens read back (two operators: what a
             prompt that arrives in pieces needs before its next piece attends)
  norm_rope  queries and keys normalised per head and rotated by position, one
             or several axes, into tensors or (keys, with the values) into a cache

A cached row is 144 bytes: 128 codes of K, 128 of V (4 bits each, sign and one of
0, 0.5, 1, 1.5, 2, 3, 4, 6), then a scale for every 16 of them: 8 of K, 8 of V. A
scale is a byte of 5 exponent and 3 mantissa bits (the upper half of an fp16
number behind its sign): the largest magnitude / 6, rounded to nearest.

``run`` computes them in plain torch operations in 32 bits, or, with ``own``
set, through the package's entry points; ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
D = 128
ROW = 144  # bytes of a cached row
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 10240.0  # 6 x this is still an fp16 number


# --------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = dict(op=op, B=4, Hq=8, Hkv=2, page=16, lo=17, hi=256, q_len=1, layout="NHD", rot=128,
             interleaved=False, axes=1, cached=True)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # a chat or two in an interactive session: latency counts
        _case("attn", "attn_small"),
        # a serving step of 64 sequences
        _case("attn", "attn_serving", B=64, Hq=32, Hkv=8, lo=512, hi=4096),
        # a few long contexts
        _case("attn", "attn_long", B=8, Hq=32, Hkv=8, page=64, lo=32768, hi=131072),
        # a serving step that verifies four drafted tokens per sequence
        _case("attn", "attn_verify", B=64, Hq=32, Hkv=8, lo=512, hi=4096, q_len=4, layout="HND"),
        # all query heads on one kv head
        _case("attn", "attn_one_kv_head", B=32, Hq=32, Hkv=1, page=64, lo=1000, hi=8000),
        # one token more for a few short sequences, handed over as bf16
        _case("cache", "cache_small"),
        # the next pieces of eight prompts, and what they attend to
        _case("cache", "cache_chunk", B=8, Hkv=8, lo=2048, hi=8192, q_len=512),
        # whole prompts
        _case("cache", "cache_prompt", B=4, Hkv=8, page=64, lo=9000, hi=16384, q_len=16384,
              layout="HND"),
        # the step before attention, for a few sequences, into their cache
        _case("norm_rope", "norm_step_small"),
        # the same for a serving step, three drafted tokens each
        _case("norm_rope", "norm_step_serving", B=64, Hq=32, Hkv=8, lo=512, hi=4096, q_len=4),
        # a long prompt
        _case("norm_rope", "norm_prompt", B=1, Hq=32, Hkv=8, q_len=16384, lo=16384, hi=16384,
              cached=False),
        # the tokens of a few images and clips: time, height and width
        _case("norm_rope", "norm_images", B=5, Hq=16, Hkv=4, q_len=1223, lo=1223, hi=1223, axes=3,
              cached=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "cache", "cache", "norm_rope", "norm_rope"])
    Hq, Hkv = rng.choice([(8, 2), (32, 8), (64, 8), (32, 1), (8, 8), (16, 4), (12, 6), (5, 1),
                          (40, 8)])
    c = dict(Hq=Hq, Hkv=Hkv, page=rng.choice([16, 32, 48, 64, 128]),
             layout=rng.choice(["NHD", "HND"]))
    if op == "attn":
        c["q_len"] = rng.choice([1, 1, 1, 1, 2, 3, 5, 8])
        hi = max(_log_int(rng, 20, 100000), c["q_len"])
        # at most the tokens x kv heads of a full serving step, and the products
        # of its verification
        most = min(64 * 4096 * 8 // (hi * Hkv), 64 * 4096 * 32 * 4 // (hi * Hq * c["q_len"]))
    elif op == "cache":
        hi = _log_int(rng, 20, 16384)
        c["q_len"] = min(hi, _log_int(rng, 1, 16384))
        most = 4 * 16384 * 8 // (hi * Hkv)
    else:
        c["cached"] = rng.random() < 0.5
        c["rot"] = rng.choice([128, 128, 128, 64, 32, 96])
        c["interleaved"] = rng.random() < 0.4
        c["axes"] = rng.choice([1, 1, 3, 2])
        c["q_len"] = _log_int(rng, 1, 64 if c["cached"] else 16384)
        hi = max(c["q_len"], _log_int(rng, 20, 8192)) if c["cached"] else c["q_len"]
        most = min(16384 * 40 // (c["q_len"] * (Hq + Hkv)), 64 * 4096 * 8 // (hi * Hkv))
    c["hi"], c["lo"] = hi, max(rng.randint(max(1, hi // 8), hi), 1 if op == "cache" else c["q_len"])
    c["B"] = max(1, min(_log_int(rng, 1, 64), most))
    return _case(op, **c)


# ------------------------------------------------------------------ structure
def _lens(c):
    """Lengths of the sequences: fixed by the case (the work depends on them)."""
    g = np.random.default_rng([c["B"], c["lo"], c["hi"]])
    lens = g.integers(c["lo"], c["hi"], size=c["B"], endpoint=True)
    lens[0] = c["hi"]
    return lens.astype(np.int64)


def _new_lens(c):
    """New tokens of each sequence (cache): at most q_len and its length."""
    g = np.random.default_rng([c["B"], c["q_len"], 5])
    most = np.minimum(_lens(c), c["q_len"])
    return np.maximum(1, most - g.integers(0, most // 4 + 1))


def _inv_freq(c):
    n = c["rot"] // 2
    return 1e6 ** (-np.arange(n, dtype=np.float64) / n)


def _axis_of(c):
    """The axis that each frequency follows: a run for each, the first the shortest."""
    n, axes = c["rot"] // 2, c["axes"]
    return [0] * n if axes == 1 else sorted(min(axes - 1, (i * axes + axes // 2) // n)
                                            for i in range(n))


def _pack(k, v):
    """Rows [..., 128] of K and V in 32 bits -> [..., 144] bytes."""
    codes, scales = [], []
    for x in (k, v):
        x = x.unflatten(-1, (8, 16))
        a = x.abs()
        top = a.amax(-1)
        top = top / torch.full_like(top, 6)  # (by a plain number it would be a product with 1 / 6)
        # 3 bits behind the leading one: 2^-3 of the power of two below, at least 2^-17
        step = ((top.view(torch.int32) & 0x7F800000).view(torch.float32) * 0.125).clamp(min=2.0 ** -17)
        s = (torch.round(top / step) * step).clamp(max=TOP_SCALE)
        b = s[..., None]
        mag = ((a > 0.25 * b).to(torch.uint8) + (a >= 0.75 * b) + (a > 1.25 * b)
               + (a >= 1.75 * b) + (a > 2.5 * b) + (a >= 3.5 * b) + (a > 5.0 * b))
        mag = torch.where(b > 0, mag, torch.zeros_like(mag)) + torch.signbit(x) * 8
        mag = mag.to(torch.uint8).flatten(-2)
        codes.append(mag[..., 0::2] + mag[..., 1::2] * 16)
        scales.append((s.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8))
    return torch.cat(codes + scales, -1)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    B, Hq, Hkv, P, q_len = c["B"], c["Hq"], c["Hkv"], c["page"], c["q_len"]
    lens = _lens(c)
    s = dict(case=c, scale=1.0 / math.sqrt(D), max_len=int(lens.max()),
             err=torch.zeros(1, dtype=torch.int32, device=DEV))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    # some channels of K are much larger than the others
    loud = torch.exp(torch.randn(Hkv, D, generator=gen, device=DEV)).to(torch.bfloat16)
    pages = None
    if c["op"] != "norm_rope" or c["cached"]:
        need = (lens + P - 1) // P
        num_pages = int(math.ceil(1.25 * int(need.sum())))
        perm = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)
        width = int(need.max())
        start = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).to(DEV)
        col = torch.arange(width, device=DEV)
        ok = col[None, :] < torch.from_numpy(need).to(DEV)[:, None]
        idx = (start[:, None] + col[None, :]).clamp_(max=num_pages - 1)
        s["bt"] = torch.where(ok, perm[idx], torch.full_like(perm[idx], -1))
        s["sl"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        pages = (num_pages, P, Hkv) if c["layout"] == "NHD" else (num_pages, Hkv, P)

    if c["op"] in ("attn", "cache"):
        pool = torch.empty(*pages, ROW, dtype=torch.uint8, device=DEV)
        ld = loud if c["layout"] == "NHD" else loud[:, None]
        n = max(1, (1 << 25) // (P * Hkv * D))
        for i in range(0, pages[0], n):
            part = pool[i:i + n]
            k, v = normal(*part.shape[:3], D) * ld, normal(*part.shape[:3], D)
            part.copy_(_pack(k.float(), v.float()))
        s["pool"] = pool
    if c["op"] == "attn":
        s["q"] = normal(B, q_len, Hq, D).mul_(2.0)
        s["out"] = torch.empty(B, q_len, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, q_len, Hq, dtype=torch.float32, device=DEV)
    elif c["op"] == "cache":
        s["k_new"], s["v_new"] = normal(B, q_len, Hkv, D) * loud, normal(B, q_len, Hkv, D)
        s["new_lens"] = torch.from_numpy(_new_lens(c).astype(np.int32)).to(DEV)
        for x in ("k_out", "v_out"):
            s[x] = torch.zeros(B, s["max_len"], Hkv, D, dtype=torch.bfloat16, device=DEV)
    else:
        # the projection's output: queries, keys and values of a token side by side
        qkv = normal(B, q_len, (Hq + 2 * Hkv) * D).mul_(3.0)
        qkv = qkv.unflatten(-1, (Hq + 2 * Hkv, D))
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 2)
        s["qw"], s["kw"] = (torch.rand(2, D, generator=gen, device=DEV) + 0.5).unbind()
        s["q_out"] = torch.empty(B, q_len, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["freq"] = torch.from_numpy(_inv_freq(c)).to(DEV)
        s["axis_of"] = torch.tensor(_axis_of(c), device=DEV)
        if c["axes"] > 1:  # frames, rows and columns behind a text
            at = torch.arange(q_len, device=DEV)
            grid = torch.stack([at // 256, at // 16 % 16, at % 16])[3 - c["axes"]:]
            first = torch.randint(0, 100000, (B,), generator=gen, device=DEV)
            s["pos"] = (grid[:, None, :] + first[None, :, None]).to(torch.int32)
        elif not c["cached"]:
            first = torch.randint(0, 100000, (B,), generator=gen, device=DEV)
            s["pos"] = (torch.arange(q_len, device=DEV) + first[:, None]).to(torch.int32)
        else:  # the places in the cache
            s["pos"] = None
        if c["cached"]:
            s["k_pool"], s["v_pool"] = normal(*pages, D), normal(*pages, D)
        else:
            s["k_out"] = torch.empty(B, q_len, Hkv, D, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _tokens(pool, bt, c):
    """The mapped rows of every sequence: [B, T, Hkv, width] (T = the table's reach)."""
    x = pool if c["layout"] == "NHD" else pool.permute(0, 2, 1, 3)
    return x[bt.clamp(min=0).long()].flatten(1, 2)


def _unpack(rows):
    """[..., 144] bytes -> K, V in 32 bits."""
    table = torch.tensor(GRID + tuple(-g for g in GRID), device=DEV)
    r = []
    for codes, scales in ((rows[..., :64], rows[..., 128:136]), (rows[..., 64:128], rows[..., 136:])):
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        x = table[x.int()].unflatten(-1, (8, 16))
        s = (scales.to(torch.int16) << 7).view(torch.float16).float()
        r.append((x * s[..., None]).flatten(-2))
    return r


def _slots(s):
    """(ok, page, slot) [B, q_len] of the new tokens."""
    c = s["case"]
    n = s["new_lens"].long()[:, None] if "new_lens" in s else c["q_len"]
    i = torch.arange(c["q_len"], device=DEV)[None, :]
    at = s["sl"].long()[:, None] - n + i
    ok = (i < n).expand_as(at)
    at = torch.where(ok, at, 0)
    return ok, torch.gather(s["bt"].long(), 1, at // c["page"]), at % c["page"]


def _scatter(pool, c, ok, page, slot, rows):
    x = pool if c["layout"] == "NHD" else pool.permute(0, 2, 1, 3)
    x[page[ok], slot[ok]] = rows[ok].to(pool.dtype)


def _plain_attn(s):
    c = s["case"]
    B, q_len, Hq, _ = s["q"].shape
    Hkv = c["Hkv"]
    g = Hq // Hkv
    k, v = (x.transpose(1, 2) for x in _unpack(_tokens(s["pool"], s["bt"], c)))
    T = k.shape[2]
    t = torch.arange(T, device=DEV)
    at = s["sl"].long()[:, None] - q_len + torch.arange(q_len, device=DEV)
    sees = t[None, None, :] <= at[:, :, None]
    q = s["q"].float().view(B, q_len, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, q_len, g, T)
    x = torch.where(sees[:, None, :, None, :], x, torch.full((), -math.inf, device=DEV))
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (x - top).exp_()
    den = p.sum(-1, keepdim=True)
    lse = (top + den.log()).squeeze(-1)
    p = p / den.clamp(min=1e-38)
    v = torch.where((t[None, :] < s["sl"][:, None])[:, None, :, None], v, torch.zeros((), device=DEV))
    out = torch.matmul(p.view(B, Hkv, -1, T), v).view(B, Hkv, q_len, g, D)
    s["out"].copy_(out.permute(0, 2, 1, 3, 4).reshape(B, q_len, Hq, D))
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(B, q_len, Hq))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_cache(s):
    c = s["case"]
    _scatter(s["pool"], c, *_slots(s), _pack(s["k_new"].float(), s["v_new"].float()))
    rows = _tokens(s["pool"], s["bt"], c)[:, :s["max_len"]]
    inside = torch.arange(s["max_len"], device=DEV)[None, :] < s["sl"][:, None]
    for to, x in zip((s["k_out"], s["v_out"]), _unpack(rows)):
        to[inside] = x[inside].to(to.dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_norm_rope(s):
    c = s["case"]
    n = c["rot"] // 2
    if s["pos"] is None:
        pos = s["sl"].long()[:, None] - c["q_len"] + torch.arange(c["q_len"], device=DEV)
        pos = pos[None]
    else:
        pos = s["pos"] if s["pos"].dim() == 3 else s["pos"][None]
    angle = pos[s["axis_of"]].permute(1, 2, 0).double() * s["freq"]   # [B, q_len, n]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        if c["interleaved"]:
            a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :n], x[..., n:2 * n]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, x[..., 2 * n:]], -1).to(torch.bfloat16)

    s["q_out"].copy_(one(s["q"], s["qw"]))
    k = one(s["k"], s["kw"])
    if not c["cached"]:
        s["k_out"].copy_(k)
        return {"q": s["q_out"], "k": s["k_out"]}
    at = _slots(s)
    _scatter(s["k_pool"], c, *at, k)
    _scatter(s["v_pool"], c, *at, s["v"])
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


# ----------------------------------------------------------- the package's own
def _own(s):
    import paged_decode_attention_gqa_gb300 as zl
    c = s["case"]
    where = dict(page_size=c["page"], layout=c["layout"], err_flags=s["err"])
    if c["op"] == "attn":
        zl.decode_attn_q4(s["q"], s["pool"], s["bt"], s["sl"], scale=s["scale"], out=s["out"],
                          lse=s["lse"], max_seq_len=s["max_len"], **where)
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "cache":
        zl.kv_append_q4(s["k_new"], s["v_new"], s["pool"], s["bt"], s["sl"],
                        new_lens=s["new_lens"], **where)
        zl.kv_read_q4(s["pool"], s["bt"], s["sl"], k_out=s["k_out"], v_out=s["v_out"], **where)
        return {"k": s["k_out"], "v": s["v_out"]}
    if "rope" not in s:  # a model's own, made once
        s["rope"] = zl.Rope(_inv_freq(c), axes=_axis_of(c), interleaved=c["interleaved"])
    if not c["cached"]:
        zl.qk_norm_rope(s["q"], s["k"], rope=s["rope"], positions=s["pos"], q_weight=s["qw"],
                        k_weight=s["kw"], eps=1e-6, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    zl.qk_norm_rope(s["q"], s["k"], rope=s["rope"], positions=s["pos"], q_weight=s["qw"],
                    k_weight=s["kw"], eps=1e-6, q_out=s["q_out"], v=s["v"], k_pool=s["k_pool"],
                    v_pool=s["v_pool"], block_table=s["bt"], seq_lens=s["sl"], **where)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "cache": _plain_cache,
            "norm_rope": _plain_norm_rope}[state["case"]["op"]](state)


# --------------------------------------------------------------------- work
def work(case):
    c = dict(case)
    lens = _lens(c)
    B, Hq, Hkv, q_len, P = c["B"], c["Hq"], c["Hkv"], c["q_len"], c["page"]
    if c["op"] == "attn":
        nbytes = int(lens.sum()) * Hkv * ROW + B * q_len * Hq * (2 * 2 * D + 4)
        nbytes += int(((lens + P - 1) // P).sum()) * 4
        return {"bytes": nbytes, "flops": 4 * int(lens.sum()) * q_len * Hq * D}
    if c["op"] == "cache":
        new, all_ = int(_new_lens(c).sum()) * Hkv, int(lens.sum()) * Hkv
        return {"bytes": new * (4 * D + ROW) + all_ * (ROW + 4 * D), "flops": 0}
    T = B * q_len
    nbytes = T * (Hq + Hkv + (Hkv if c["cached"] else 0)) * 4 * D
    nbytes += 4 * (T * c["axes"] if not c["cached"] or c["axes"] > 1 else B)
    return {"bytes": nbytes, "flops": T * (Hq + Hkv) * (4 * D + 3 * c["rot"])}


# --------------------------------------------------------------------- exact
def _values64(rows):
    """[n, 144] bytes -> K, V [n, 128] in 64 bits, code by code from tables."""
    b = rows.cpu().numpy()
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    code = np.concatenate([mag, -mag])
    byte = np.arange(256)
    e, m = byte >> 3, byte & 7
    scale = np.where(e == 0, m * 2.0 ** -17, (8 + m) * 2.0 ** (e - 18.0))
    r = []
    for at, sc in ((0, 128), (64, 136)):
        x = np.empty((len(b), 8, 8, 2))
        x[..., 0] = code[b[:, at:at + 64] & 15].reshape(-1, 8, 8)
        x[..., 1] = code[b[:, at:at + 64] >> 4].reshape(-1, 8, 8)
        x *= scale[b[:, sc:sc + 8]][:, :, None, None]
        r.append(torch.from_numpy(x.reshape(-1, D)).to(DEV))
    return r


def _exact_rows(s, b, h, L):
    P = s["case"]["page"]
    t = torch.arange(L, device=DEV)
    pages, slots = s["bt"][b, t // P].long(), t % P
    return s["pool"][pages, slots, h] if s["case"]["layout"] == "NHD" else s["pool"][pages, h, slots]


def _exact_attn(s):
    c = s["case"]
    B, q_len, Hq, _ = s["q"].shape
    g = Hq // c["Hkv"]
    out = torch.zeros(B, q_len, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, q_len, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["sl"].tolist()):
        see = torch.ones(q_len, L, dtype=torch.bool, device=DEV).tril(L - q_len)
        for h in range(c["Hkv"]):
            kk, vv = _values64(_exact_rows(s, b, h, L))
            qq = s["q"][b, :, h * g:(h + 1) * g].double()
            x = torch.einsum("qgd,td->qgt", qq, kk) * s["scale"]
            x = x.masked_fill(~see[:, None, :], -math.inf)
            z = torch.logsumexp(x, 2)
            p = torch.where(torch.isinf(z)[..., None], 0.0, torch.exp(x - z[..., None]))
            out[b, :, h * g:(h + 1) * g] = torch.einsum("qgt,td->qgd", p, vv)
            lse[b, :, h * g:(h + 1) * g] = z
    return {"out": out, "lse": lse}


def _nearest64(x):
    """[..., 16] -> the values their codes and scale stand for: the scale whose 6-fold
    is nearest to the largest, then for each element the nearest of the 8 values
    (ties: the even byte or code)."""
    table = torch.tensor([(i & 7) * 2.0 ** -17 if i < 8 else (8 + (i & 7)) * 2.0 ** ((i >> 3) - 18)
                          for i in range(256)], dtype=torch.float64, device=DEV)
    table = table[table <= TOP_SCALE]
    a = x.abs()
    want = a.amax(-1)
    up = torch.searchsorted(6 * table, want).clamp(max=len(table) - 1)
    down = (up - 1).clamp(min=0)
    du, dd = (6 * table[up] - want).abs(), (want - 6 * table[down]).abs()
    take_up = (du < dd) | ((du == dd) & (up % 2 == 0))
    s = torch.where(take_up, table[up], table[down])[..., None]
    best = torch.zeros_like(a)
    gap = a.clone()                                  # code 0
    for g in (1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0):    # even codes, then odd ones
        d = (a - g * s).abs()
        closer = d < gap
        best, gap = torch.where(closer, g * s, best), torch.where(closer, d, gap)
    return torch.copysign(best, x)


def _exact_cache(s):
    c = s["case"]
    k, v = s["k_out"].double(), s["v_out"].double()
    for b, (L, n) in enumerate(zip(s["sl"].tolist(), s["new_lens"].tolist())):
        for h in range(c["Hkv"]):
            k[b, :L, h], v[b, :L, h] = _values64(_exact_rows(s, b, h, L))
        for to, x in ((k, s["k_new"]), (v, s["v_new"])):
            to[b, L - n:L] = _nearest64(x[b, :n].double().unflatten(-1, (8, 16))).flatten(-2)
    return {"k": k, "v": v}


def _exact_norm_rope(s):
    c = s["case"]
    n, q_len = c["rot"] // 2, c["q_len"]
    if s["pos"] is None:
        pos = torch.stack([torch.arange(L - q_len, L) for L in s["sl"].tolist()]).to(DEV)[None]
    else:
        pos = s["pos"].reshape(c["axes"], c["B"], q_len)
    turn = torch.stack([pos[a].double() * f for a, f in zip(_axis_of(c), _inv_freq(c))], -1)
    turn = torch.polar(torch.ones_like(turn), turn)[:, :, None]

    def one(x, w):
        x = x.double()
        x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6)
        pair = (torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if c["interleaved"]
                else torch.complex(x[..., :n], x[..., n:2 * n])) * turn
        x = x.clone()
        if c["interleaved"]:
            x[..., 0:2 * n:2], x[..., 1:2 * n:2] = pair.real, pair.imag
        else:
            x[..., :n], x[..., n:2 * n] = pair.real, pair.imag
        return x

    q, k = one(s["q"], s["qw"]), one(s["k"], s["kw"])
    if not c["cached"]:
        return {"q": q, "k": k}
    pools = []
    for pool, rows in ((s["k_pool"].double(), k), (s["v_pool"].double(), s["v"].double())):
        for b, L in enumerate(s["sl"].tolist()):
            for i in range(q_len):
                t = L - q_len + i
                page, slot = int(s["bt"][b, t // c["page"]]), t % c["page"]
                if c["layout"] == "NHD":
                    pool[page, slot] = rows[b, i]
                else:
                    pool[page, :, slot] = rows[b, i]
        pools.append(pool)
    return {"q": q, "k_pool": pools[0], "v_pool": pools[1]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "cache": _exact_cache,
            "norm_rope": _exact_norm_rope}[case["op"]](s)
