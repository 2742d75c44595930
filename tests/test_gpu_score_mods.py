"""Decode attention with modified scores on the GPU against the plain 64-bit
form: tanh cap, distance bias, window, drafted trees, accumulated weights."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from paged_decode_attention_gqa_gb300 import workloads as wl
from plain_ops import attention, check, f64

pytestmark = pytest.mark.gpu


def nhd(w, pool):
    return f64(pool if w.layout == "NHD" else pool.permute(0, 2, 1, 3))


def random_trees(g, B, q_len):
    par = np.full((B, q_len), -1)
    for b in range(B):
        for i in range(1, q_len):
            par[b, i] = g.integers(-1, i)
    return zl.tree_mask(par)


def run(w, *, block_table=None, seq_lens=None, softcap=0.0, slopes=None, window=0, mask=None,
        weights=None, decay=1.0, max_seq_len=0, num_ctas=0, q_scale=None, expect_bad=None):
    """One call against the plain form; returns (out, lse, weights) on the GPU."""
    bt = w.block_table if block_table is None else block_table
    sl = w.seq_lens if seq_lens is None else seq_lens
    dev = "cuda"
    out = torch.full((w.B, w.q_len, w.Hq, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full((w.B, w.q_len, w.Hq), float("nan"), device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    wg = None if weights is None else weights.clone().to(dev)
    zl.decode_attn(w.q.to(dev), w.k_pool.to(dev), w.v_pool.to(dev), torch.from_numpy(bt).to(dev),
                   torch.from_numpy(sl).to(dev), page_size=w.page_size, scale=w.scale, out=out,
                   lse=lse, err_flags=err, layout=w.layout, softcap=softcap,
                   alibi_slopes=None if slopes is None else slopes.to(dev), window=window,
                   tree_mask=None if mask is None else mask.to(dev), weights=wg,
                   weights_decay=decay, max_seq_len=max_seq_len, num_ctas=num_ctas)
    torch.cuda.synchronize()
    ref = attention(f64(w.q), nhd(w, w.k_pool), nhd(w, w.v_pool), bt, sl, scale=w.scale,
                    softcap=softcap, slopes=None if slopes is None else f64(slopes),
                    window=window, mask=mask, tokens=None if weights is None else weights.shape[2],
                    num_pages=w.num_pages, decay=decay,
                    old=None if weights is None else f64(weights))
    assert int(err.item()) == ref.bad == (expect_bad or 0)
    check(f64(out), ref.out, ref.out_tol, "out")
    check(f64(lse), ref.lse, ref.lse_tol, "lse")
    if wg is not None:
        check(f64(wg), ref.weights, ref.weights_tol, "weights")
    return out, lse, wg


def slopes_of(Hq):
    return 2.0 ** (-8.0 * (torch.arange(Hq, dtype=torch.float32) + 1) / Hq)


MODS = {
    "cap": dict(softcap=3.0),
    "alibi": dict(slopes=True),
    "window": dict(window=40),
    "window1": dict(window=1),
    "all": dict(softcap=20.0, slopes=True, window=100),
}


def mods_of(name, Hq):
    m = dict(MODS[name])
    if m.get("slopes"):
        m["slopes"] = slopes_of(Hq)
    return m


@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, 1), (8, 8, 3), (32, 8, 2), (5, 1, 1), (32, 1, 1),
                                          (12, 6, 7), (40, 8, 5)])
def test_mods_heads_and_tokens(mod, Hq, Hkv, q_len):
    w = wl.random_case(2000 + Hq + q_len, B=4, Hq=Hq, Hkv=Hkv, q_len=q_len,
                       lens=[max(q_len, 1), 17, 130, 300])
    run(w, **mods_of(mod, Hq))


@pytest.mark.parametrize("P,layout", [(16, "HND"), (32, "NHD"), (48, "NHD"), (64, "HND"),
                                      (128, "NHD")])
def test_mods_pages_and_layouts(P, layout):
    w = wl.random_case(2100 + P, B=5, Hq=16, Hkv=4, page_size=P, layout=layout,
                       lens=[1, P - 1, P, P + 1, 3 * P + 5])
    run(w, **mods_of("all", 16))
    run(w, window=P // 2)


@pytest.mark.parametrize("msl", [0, 400])
@pytest.mark.parametrize("ctas", [0, 1, 3, 40])
def test_mods_any_split(ctas, msl):
    w = wl.random_case(2200, B=3, Hq=8, Hkv=2, lens=[400, 33, 0], q_len=2)
    run(w, num_ctas=ctas, max_seq_len=msl, **mods_of("all", 8))


def test_cap_saturates():
    """Scores far beyond the cap: tanh is at +-1 and ties share the weight."""
    w = wl.random_case(2210, B=2, Hq=4, Hkv=2, lens=[64, 200])
    w.q *= 100
    run(w, softcap=2.0)


def test_long_distance_bias():
    """A steep bias over a long context: old tokens vanish, near ones are exact."""
    w = wl.random_case(2220, B=1, Hq=8, Hkv=2, lens=[5000], page_size=64)
    run(w, slopes=torch.linspace(0.001, 1.0, 8))
    run(w, slopes=-torch.linspace(0.0, 0.01, 8))  # towards the old ones


@pytest.mark.parametrize("q_len", [2, 3, 8, 16, 33, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (32, 1)])
def test_trees(q_len, Hq, Hkv):
    w = wl.random_case(2300 + q_len, B=3, Hq=Hq, Hkv=Hkv, q_len=q_len,
                       lens=[q_len, q_len + 50, 300])
    mask = random_trees(np.random.default_rng(q_len), 3, q_len)
    run(w, mask=mask)


@pytest.mark.parametrize("mod", ["cap", "alibi", "window", "window1", "all"])
@pytest.mark.parametrize("q_len", [5, 40])
def test_trees_with_mods(mod, q_len):
    w = wl.random_case(2400, B=3, Hq=8, Hkv=2, q_len=q_len, lens=[q_len, 70, 290], layout="HND",
                       page_size=32)
    run(w, mask=random_trees(np.random.default_rng(7), 3, q_len), **mods_of(mod, 8))


@pytest.mark.parametrize("q_len", [4, 48])
def test_tree_rows_without_tokens(q_len):
    """Empty masks with no context: zeros and -inf; empty masks with context see
    only that; arbitrary bits are taken as they are; fewer tokens than drafted."""
    w = wl.random_case(2410, B=4, Hq=8, Hkv=2, q_len=q_len, lens=[q_len, q_len + 30, q_len - 2, 0])
    mask = torch.zeros(4, q_len, (q_len + 31) // 32, dtype=torch.int32)
    out, lse, _ = run(w, mask=mask)
    assert torch.isinf(lse[0]).all() and (out[0] == 0).all()
    g = torch.Generator().manual_seed(1)
    bits = torch.randint(0, 2, (4, q_len, q_len), generator=g)
    words = torch.zeros_like(mask, dtype=torch.int64)
    for j in range(q_len):
        words[:, :, j // 32] |= bits[:, :, j].long() << (j % 32)
    mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    run(w, mask=mask)
    run(w, mask=mask, window=9, slopes=slopes_of(8))


@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, 1), (32, 8, 1), (32, 1, 1), (5, 1, 3), (4, 4, 9),
                                          (8, 2, 20)])
@pytest.mark.parametrize("mod", [None, "all", "window"])
@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
def test_weights(Hq, Hkv, q_len, mod, decay):
    w = wl.random_case(2500, B=4, Hq=Hq, Hkv=Hkv, q_len=q_len, lens=[q_len, 63, 300, 0])
    old = torch.rand(4, Hkv, 320, generator=torch.Generator().manual_seed(3))
    if decay == 0.0:
        old[:, :, ::2] = float("nan")   # old values do not count
    run(w, weights=old, decay=decay, **(mods_of(mod, Hq) if mod else {}))


def test_weights_with_trees_and_strides():
    w = wl.random_case(2510, B=3, Hq=8, Hkv=2, q_len=6, lens=[6, 80, 200])
    mask = random_trees(np.random.default_rng(5), 3, 6)
    run(w, mask=mask, weights=torch.zeros(3, 2, 200))
    # rows inside a larger buffer, token rows 7 elements apart from alignment
    big = torch.rand(3, 4, 333, device="cuda")
    keep = big.clone()
    view = big[:, 1:3, 7:307]
    args = dict(page_size=16, scale=w.scale, tree_mask=mask.cuda())
    ins = [x.cuda() for x in (w.q, w.k_pool, w.v_pool, torch.from_numpy(w.block_table),
                              torch.from_numpy(w.seq_lens))]
    zl.decode_attn(*ins, weights=view, **args)
    plain = keep[:, 1:3, 7:307].contiguous()
    zl.decode_attn(*ins, weights=plain, **args)
    assert torch.equal(view, plain)
    assert torch.equal(big[:, 0], keep[:, 0]) and torch.equal(big[:, 3], keep[:, 3])
    assert torch.equal(big[:, :, :7], keep[:, :, :7]) and torch.equal(big[:, :, 307:],
                                                                      keep[:, :, 307:])


def test_weights_rows_too_short_flag_the_sequence():
    w = wl.random_case(2520, B=3, Hq=8, Hkv=2, lens=[60, 100, 64])
    run(w, weights=torch.rand(3, 2, 64), expect_bad=zl.DEVERR_BAD_SEQ_LEN)


def test_weights_sum_to_the_query_rows():
    """Each query row's weights sum to 1 over the tokens."""
    w = wl.random_case(2530, B=2, Hq=32, Hkv=8, lens=[1000, 2000])
    _, _, wg = run(w, weights=torch.zeros(2, 8, 2000))
    s = wg.double().sum(2).cpu()
    # 4 rows; each weight within 2^-20, fp32 sum of l over 2000 tokens
    assert ((s - 4.0).abs() < 4 * 2000 / 16 * 2.0 ** -24 + 4 * 2.0 ** -18).all()


@pytest.mark.parametrize("q_len,kw", [(1, dict(softcap=5.0)), (6, dict(tree=True)),
                                      (40, dict(tree=True)), (1, dict(weights=True)),
                                      (3, dict(window=50))])
def test_bad_pages_and_lengths(q_len, kw):
    kw = dict(kw)
    w = wl.random_case(2600, B=6, Hq=8, Hkv=2, q_len=q_len, lens=[100, 90, 200, 64, 150, 80],
                       poison=False)
    bt, sl = w.block_table.copy(), w.seq_lens.copy()
    bt[0, 2] = w.num_pages          # rows that see tokens 32..47
    bt[2, (200 - 1) // 16] = -5     # the newest tokens' page
    bt[3, 0] = 1 << 30
    sl[4] = -1
    sl[5] = bt.shape[1] * 16 + 1
    if kw.pop("tree", None):
        kw["mask"] = random_trees(np.random.default_rng(2), 6, q_len)
    if kw.pop("weights", None):
        kw["weights"] = torch.rand(6, 2, 220)
    run(w, block_table=bt, seq_lens=sl, expect_bad=3, **kw)


def test_window_pages_need_not_be_mapped():
    """Pages wholly before the window may be unmapped, and hold NaN."""
    for q_len in (1, 4, 24):
        w = wl.random_case(2610, B=3, Hq=8, Hkv=2, q_len=q_len, lens=[500, 300, 250])
        bt = w.block_table.copy()
        k, v = w.k_pool, w.v_pool
        for b, L in enumerate(w.seq_lens):
            lo = L - q_len - 60 + 1
            for j in range(lo // 16):
                k[bt[b, j]], v[bt[b, j]] = float("nan"), float("nan")
                if b != 1:
                    bt[b, j] = -1
            k[bt[b, lo // 16], :lo % 16] = float("nan")
            v[bt[b, lo // 16], :lo % 16] = float("nan")
        # the plain form reads the same pools: NaN where it does not look
        run(w, block_table=bt, window=60)


@pytest.mark.parametrize("q_len,Hq,Hkv", [(1, 32, 8), (16, 8, 2), (64, 8, 2)])
def test_page_remap_and_repeat_are_bit_identical(q_len, Hq, Hkv):
    w = wl.random_case(2620, B=4, Hq=Hq, Hkv=Hkv, q_len=q_len, lens=[300, 150, 700, q_len])
    mask = random_trees(np.random.default_rng(4), 4, q_len)
    kw = dict(softcap=10.0, mask=mask, weights=torch.zeros(4, Hkv, 720))
    a = run(w, **kw)
    again = run(w, **kw)
    perm = np.random.default_rng(1).permutation(w.num_pages)
    w2 = wl.random_case(2620, B=4, Hq=Hq, Hkv=Hkv, q_len=q_len, lens=[300, 150, 700, q_len])
    inv = torch.from_numpy(np.argsort(perm))
    w2.k_pool, w2.v_pool = w.k_pool[inv], w.v_pool[inv]
    bt = w.block_table.copy()
    bt[bt >= 0] = perm[bt[bt >= 0]]
    w2.block_table = bt.astype(np.int32)
    b = run(w2, **kw)
    for x, y, z in zip(a, again, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal(x.view(torch.uint8), z.view(torch.uint8))


@pytest.mark.parametrize("q_len,layout", [(1, "NHD"), (3, "HND"), (24, "NHD")])
def test_fused_append(q_len, layout):
    """k_new / v_new with modified scores: the pools and the output of a
    separate append followed by the call."""
    w = wl.random_case(2700, B=4, Hq=8, Hkv=2, q_len=q_len, lens=[q_len, 60, 200, 333],
                       layout=layout)
    kn, vn = (x.cuda() for x in wl.new_token_rows(2700, 4, q_len, 2, 128, 128))
    bt, sl = torch.from_numpy(w.block_table).cuda(), torch.from_numpy(w.seq_lens).cuda()
    got = []
    for fused in (False, True):
        k, v = w.k_pool.cuda(), w.v_pool.cuda()
        if not fused:
            zl.kv_append(kn, vn, k, v, bt, sl, page_size=16, layout=layout)
        out = zl.decode_attn(w.q.cuda(), k, v, bt, sl, page_size=16, scale=w.scale, softcap=9.0,
                             window=120, layout=layout, **(dict(k_new=kn, v_new=vn) if fused else {}))
        torch.cuda.synchronize()
        got.append((out, k, v))
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("q_len", [1, 24])
def test_graph_replay_and_other_stream(q_len):
    """Two captured graphs, replayed on two streams at once, and an eager call on
    a stream that is not the current one: each its own scratch."""
    w = wl.random_case(2710, B=4, Hq=8, Hkv=2, q_len=q_len, lens=[300, 200, 100, 700])
    ins = [x.cuda() for x in (w.q, w.k_pool, w.v_pool, torch.from_numpy(w.block_table),
                              torch.from_numpy(w.seq_lens))]
    kw = dict(page_size=16, scale=w.scale, softcap=4.0)
    wsum = torch.zeros(4, 2, 700, device="cuda")
    want = zl.decode_attn(*ins, weights=wsum, **kw)
    alone = zl.decode_attn(*ins, **kw)  # (many rows without weights: another kernel)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g, wt = torch.cuda.CUDAGraph(), torch.zeros(4, 2, 700, device="cuda")
        with torch.cuda.graph(g):
            o = zl.decode_attn(*ins, weights=wt, weights_decay=0.0, **kw)
        graphs.append((g, o, wt))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = zl.decode_attn(*ins, stream=side, **kw)
    torch.cuda.synchronize()
    for _, o, wt in graphs:
        assert bool(torch.equal(o.view(torch.int16), want.view(torch.int16)))
        assert bool(torch.equal(wt, wsum))
    assert bool(torch.equal(eager.view(torch.int16), alone.view(torch.int16)))


def test_plain_call_is_the_unmodified_path():
    """softcap 0, window 0 and no tensors run zl_decode_attn, bit for bit."""
    w = wl.random_case(2720, B=3, Hq=8, Hkv=2, lens=[30, 200, 77])
    ins = [x.cuda() for x in (w.q, w.k_pool, w.v_pool, torch.from_numpy(w.block_table),
                              torch.from_numpy(w.seq_lens))]
    a = zl.decode_attn(*ins, page_size=16, scale=w.scale)
    b = zl.decode_attn(*ins, page_size=16, scale=w.scale, softcap=0.0, window=0)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_far_pages_and_large_batch():
    """Pages beyond 2^31 elements of the pool, and more sequences than the small
    tile table holds."""
    pages = (1 << 31) // (16 * 2 * 128) + 64
    k = torch.zeros(pages, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for q_len in (1, 20):
        lens = [70, 45]
        bt = torch.tensor([[pages - 1, pages - 7, 3, pages - 20, pages - 2],
                           [pages - 9, pages - 30, pages - 31, 0, 0]], dtype=torch.int32)
        used = bt.flatten().unique().long()
        k[used.cuda()] = torch.randn(len(used), 16, 2, 128, generator=g, device="cuda").bfloat16()
        v[used.cuda()] = torch.randn(len(used), 16, 2, 128, generator=g, device="cuda").bfloat16()
        q = torch.randn(2, q_len, 8, 128, generator=g, device="cuda").bfloat16()
        out = zl.decode_attn(q, k, v, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             page_size=16, scale=0.1, softcap=8.0)
        small = {int(p): i for i, p in enumerate(used)}
        sbt = np.array([[small[int(x)] for x in row] for row in bt], dtype=np.int32)
        ref = attention(f64(q), f64(k[used.cuda()]), f64(v[used.cuda()]), sbt, lens, scale=0.1,
                        softcap=8.0)
        check(f64(out), ref.out, ref.out_tol, "out")
    del k, v
    w = wl.random_case(2730, B=600, Hq=4, Hkv=2, max_len=40)
    run(w, softcap=6.0, window=20)


# Calls of many query rows per kv head: another kernel, whose tiles are
# 128 tokens wide and 128 rows high.


@pytest.mark.parametrize("P,layout", [(16, "HND"), (32, "NHD"), (48, "NHD"), (48, "HND"),
                                      (64, "HND"), (128, "NHD"), (256, "HND")])
def test_many_rows_pages_and_layouts(P, layout):
    w = wl.random_case(2800 + P, B=5, Hq=16, Hkv=4, page_size=P, layout=layout, q_len=12,
                       lens=[12, P - 1, P, P + 1, 3 * P + 5])
    mask = random_trees(np.random.default_rng(P), 5, 12)
    run(w, **mods_of("all", 16))
    run(w, mask=mask, **mods_of("all", 16))
    run(w, mask=mask, window=P // 2 + 3)


@pytest.mark.parametrize("Hq,Hkv,q_len", [(128, 1, 1), (128, 1, 5), (64, 1, 4), (5, 1, 60),
                                          (24, 2, 7), (7, 7, 90), (33, 1, 9), (100, 1, 3),
                                          (9, 3, 128)])
@pytest.mark.parametrize("tree", [False, True])
def test_many_rows_heads(Hq, Hkv, q_len, tree):
    w = wl.random_case(2810, B=3, Hq=Hq, Hkv=Hkv, q_len=q_len,
                       lens=[max(q_len, 1), q_len + 130, 700])
    mask = random_trees(np.random.default_rng(3), 3, q_len) if tree else None
    run(w, mask=mask, softcap=4.0, slopes=slopes_of(Hq))


@pytest.mark.parametrize("ctx", [0, 1, 31, 63, 64, 65, 90, 127, 128, 129, 190, 255, 256])
@pytest.mark.parametrize("q_len", [33, 64, 65, 128])
def test_drafted_tokens_across_tiles(ctx, q_len):
    """Every place of the first drafted token in its tile: the distance bias and
    the window go by depth there, not by place."""
    w = wl.random_case(2820 + ctx, B=2, Hq=2, Hkv=2, q_len=q_len, lens=[ctx + q_len] * 2)
    mask = random_trees(np.random.default_rng(ctx), 2, q_len)
    run(w, mask=mask, slopes=torch.tensor([0.3, 0.01]))
    run(w, mask=mask, slopes=torch.tensor([0.3, 0.01]), window=5, softcap=3.0)
    # a chain, whose depths are the places
    chain = zl.tree_mask(np.tile(np.arange(q_len) - 1, (2, 1)))
    a = run(w, mask=chain, slopes=torch.tensor([0.3, 0.01]), window=70)
    b = run(w, slopes=torch.tensor([0.3, 0.01]), window=70)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))


@pytest.mark.parametrize("ctas", [0, 1, 2, 7, 60, 152])
@pytest.mark.parametrize("q_len,Hq,Hkv", [(20, 8, 2), (50, 32, 1)])
def test_many_rows_any_split(ctas, q_len, Hq, Hkv):
    w = wl.random_case(2830, B=4, Hq=Hq, Hkv=Hkv, lens=[4000, 33, 0, 900], q_len=q_len,
                       page_size=32, values=True)
    mask = random_trees(np.random.default_rng(8), 4, q_len)
    for msl in (0, 4000):
        run(w, num_ctas=ctas, max_seq_len=msl, mask=mask, **mods_of("alibi", Hq))


def test_many_rows_many_sequences():
    w = wl.random_case(2840, B=700, Hq=4, Hkv=1, max_len=60, q_len=12)
    run(w, softcap=6.0, window=20)
    run(w, mask=random_trees(np.random.default_rng(8), 700, 12))
    # whole units, several to a CTA, some of them empty; then one that is too long
    g = np.random.default_rng(2)
    lens = g.integers(0, 500, size=300)
    lens[::7] = 0
    for last in (500, 700):
        lens[-1] = last
        w = wl.random_case(2841, B=300, Hq=8, Hkv=2, lens=lens, q_len=6)
        run(w, mask=random_trees(np.random.default_rng(8), 300, 6), slopes=slopes_of(8))


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("scale,cap", [(1e-3, 50.0), (0.09, 1e-3), (0.09, 1e4), (3.0, 50.0),
                                       (1e-30, 1.0)])
def test_caps_far_from_the_scores(q_len, scale, cap):
    w = wl.random_case(2850, B=2, Hq=4, Hkv=2, lens=[64, 200], q_len=q_len, scale=scale)
    run(w, softcap=cap)


@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 8, 1), (8, 1, 2), (4, 1, 20)])
def test_bad_pages_in_calls_of_few_rows(Hq, Hkv, q_len):
    """One sequence in many pieces, one of which meets a bad page."""
    w = wl.random_case(2860, B=1, Hq=Hq, Hkv=Hkv, q_len=q_len, lens=[9000], poison=False)
    for at in (0, 300, 9000 // 16):
        bt = w.block_table.copy()
        bt[0, at] = w.num_pages
        run(w, block_table=bt, softcap=5.0, expect_bad=1)
        run(w, block_table=bt, window=500, expect_bad=0 if at < 500 else 1)


@pytest.mark.parametrize("window", [299, 300, 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("q_len", [4, 24])
def test_windows_longer_than_any_sequence(q_len, window):
    """Nothing is hidden, also where fewer tokens are cached than drafted."""
    w = wl.random_case(2870, B=4, Hq=8, Hkv=2, q_len=q_len, lens=[1, q_len - 1, 300, 150])
    run(w, window=window)
    mask = random_trees(np.random.default_rng(1), 4, q_len)
    run(w, window=window, mask=mask, weights=torch.zeros(4, 2, 300))


@pytest.mark.parametrize("Hq,Hkv,q_len,ctas,msl,weights", [
    (8, 2, 1, 0, 0, False), (8, 2, 1, 1000, 0, True), (32, 8, 2, 0, 400, True),
    (32, 1, 1, 0, 0, True), (8, 2, 24, 0, 0, False), (8, 2, 24, 700, 0, False),
    (32, 1, 24, 3, 0, False), (8, 2, 24, 0, 400, False), (32, 2, 20, 0, 0, True)])
def test_explicit_workspace_of_the_exact_size(Hq, Hkv, q_len, ctas, msl, weights):
    """The parameter structs and a workspace of the caller's: the bytes asked for
    suffice, none past them are touched, and one byte less is refused."""
    w = wl.random_case(2880, B=4, Hq=Hq, Hkv=Hkv, q_len=q_len, lens=[400, 130, 0, 257])
    q, k, v, bt, sl = (x.cuda() for x in (w.q, w.k_pool, w.v_pool,
                                          torch.from_numpy(w.block_table),
                                          torch.from_numpy(w.seq_lens)))
    mods = dict(softcap=6.0, alibi_slopes=slopes_of(Hq).cuda(), window=300,
                tree_mask=random_trees(np.random.default_rng(3), 4, q_len).cuda())
    wa = torch.zeros(4, Hkv, 400, device="cuda") if weights else None
    wb = None if wa is None else wa.clone()
    call = dict(page_size=16, scale=w.scale, num_ctas=ctas, max_seq_len=msl)
    want = zl.decode_attn(q, k, v, bt, sl, weights=wa, **call, **mods)
    out = torch.empty_like(want)
    p = zl.make_params(q, k, v, bt, sl, out, Hkv=Hkv, D_v=128, **call)
    m = zl.make_score_params(q, Hkv, weights=wb, **mods)
    n = zl.workspace_size_ex(p, m)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    p.workspace, p.workspace_bytes = buf.data_ptr(), n
    zl.call_ex(p, m)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    if weights:
        assert torch.equal(wa, wb)
    assert bool((buf[n:] == 0xA5).all())
    if n:
        p.workspace_bytes = n - 1
        with pytest.raises(zl.ZlError):
            zl.call_ex(p, m)
