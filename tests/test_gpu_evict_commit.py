"""Eviction by accumulated weights and commit of a drafted path on the GPU: the
moved rows, weights, lists and lengths equal the plain form's exactly, and the
operators run together as a decode loop runs them."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from paged_decode_attention_gqa_gb300 import workloads as wl
from plain_ops import attention, check, commit, evict, f64

pytestmark = pytest.mark.gpu


def u16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def cuda(*ts):
    return [None if t is None else (torch.from_numpy(t) if isinstance(t, np.ndarray) else t).cuda()
            for t in ts]


def nhd(w, t):
    return None if t is None else (t if w.layout == "NHD" else t.permute(0, 2, 1, 3))


def run_evict(w, weights, *, budget, sink=0, recent=0, dst=None, weights_out=None,
              block_table=None, seq_lens=None, expect=0):
    bt = w.block_table if block_table is None else block_table
    sl = w.seq_lens if seq_lens is None else seq_lens
    k, v, wg, btd, sld, dstd, wod = cuda(w.k_pool.clone(), None if w.v_pool is None
                                         else w.v_pool.clone(), weights.clone(), bt, sl, dst,
                                         None if weights_out is None else weights_out.clone())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.full((w.B, w.Hkv, budget), 77, dtype=torch.int32, device="cuda")
    new, kept = zl.kv_evict(k, v, btd, sld, wg, page_size=w.page_size, budget=budget, sink=sink,
                            recent=recent, dst_block_table=dstd, weights_out=wod, kept=kept,
                            layout=w.layout, err_flags=err)
    torch.cuda.synchronize()
    ref = evict(u16(nhd(w, w.k_pool)), None if w.v_pool is None else u16(nhd(w, w.v_pool)),
                weights.numpy(), bt, sl, page_size=w.page_size, budget=budget, sink=sink,
                recent=recent, num_pages=w.num_pages, dst_table=dst,
                weights_out=None if weights_out is None else weights_out.numpy())
    rk, rv, rw, rkept, rnew, rerr = ref
    assert int(err.item()) == rerr == expect
    assert np.array_equal(kept.cpu().numpy(), rkept)
    assert np.array_equal(new.cpu().numpy(), rnew)
    got_w = (wg if wod is None else wod).cpu().numpy()
    assert np.array_equal(got_w.view(np.uint32), rw.view(np.uint32))
    if wod is not None:
        assert torch.equal(wg.cpu().view(torch.int32), weights.view(torch.int32))
    assert np.array_equal(u16(nhd(w, k)), rk)
    if v is not None:
        assert np.array_equal(u16(nhd(w, v)), rv)
    return new, kept


def weights_for(w, T, seed, kind="spread"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(w.B, w.Hkv, T, generator=g).mul(2).exp()
    if kind == "ties":
        x = torch.randint(0, 4, x.shape, generator=g).float()
    if kind == "equal":
        x = torch.full_like(x, 0.25)
    if kind == "odd":  # every kind of value a float can hold
        vals = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-42, -1.0,
                             3.4e38, 1.0])
        x = vals[torch.randint(0, len(vals), x.shape, generator=g)]
    return x


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("budget,sink,recent", [(64, 0, 0), (64, 4, 16), (50, 7, 43), (1, 0, 0),
                                                (33, 0, 33), (33, 33, 0), (299, 1, 2)])
def test_evict_in_place(kind, budget, sink, recent):
    w = wl.random_case(3100, B=6, Hq=8, Hkv=2, lens=[300, 1, 0, 64, 65, 150])
    run_evict(w, weights_for(w, 310, budget, kind), budget=budget, sink=sink, recent=recent)


@pytest.mark.parametrize("Hkv,P,layout", [(1, 16, "NHD"), (8, 32, "HND"), (3, 48, "NHD"),
                                          (4, 128, "HND")])
def test_evict_pages_and_layouts(Hkv, P, layout):
    w = wl.random_case(3110 + P, B=3, Hq=2 * Hkv, Hkv=Hkv, page_size=P, layout=layout,
                       lens=[2 * P + 1, 900, 400])
    run_evict(w, weights_for(w, 900, 1), budget=300, sink=3, recent=50)


@pytest.mark.parametrize("B,Hkv,L,budget", [(1, 1, 20000, 15001), (1, 2, 9000, 2500),
                                            (2, 8, 5000, 4999)])
def test_evict_long(B, Hkv, L, budget):
    """More rows than one look-up of places, few blocks (narrow column parts)."""
    w = wl.random_case(3120, B=B, Hq=Hkv, Hkv=Hkv, page_size=64, lens=[L] * B)
    run_evict(w, weights_for(w, L, 2), budget=budget, sink=4, recent=budget // 3)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
def test_evict_rows_beyond_the_registers_of_a_cluster(kind):
    """Rows of more than 131072 weights are read anew for each step of the search."""
    w = wl.random_case(3125, B=3, Hq=1, Hkv=1, page_size=128, lens=[140000, 131073, 300],
                       poison=False)
    wt = weights_for(w, 140003, 9, kind)
    run_evict(w, wt, budget=4097, sink=4, recent=1000)
    free = np.setdiff1d(np.arange(w.num_pages), w.block_table[w.block_table >= 0])
    dst = free[:3 * 33].reshape(3, 33).astype(np.int32)
    run_evict(w, wt, budget=4097, recent=30, dst=dst)


def test_evict_into_new_pages():
    w = wl.random_case(3130, B=4, Hq=8, Hkv=2, lens=[700, 120, 33, 0], pool_factor=3.0)
    free = np.setdiff1d(np.arange(w.num_pages), w.block_table[w.block_table >= 0])
    dst = np.full((4, 9), -1, dtype=np.int32)
    dst.flat[:] = free[:36]
    wt = weights_for(w, 705, 3)
    run_evict(w, wt, budget=130, sink=2, recent=20, dst=dst)
    run_evict(w, wt, budget=130, sink=2, recent=20, dst=dst, weights_out=torch.zeros(4, 2, 130))
    run_evict(w, wt, budget=130, sink=2, recent=20, weights_out=torch.zeros(4, 2, 140))


def test_evict_latent_pool():
    w = wl.random_case(3140, B=3, Hq=128, Hkv=1, D=576, page_size=64, mla=True, D_v=512,
                       lens=[300, 64, 200])
    run_evict(w, weights_for(w, 300, 4), budget=100, sink=1, recent=10)


def test_evict_errors():
    w = wl.random_case(3150, B=6, Hq=8, Hkv=2, lens=[100, 90, 80, 120, 64, 110], pool_factor=3.0)
    bt, sl = w.block_table.copy(), w.seq_lens.copy()
    bt[0, 3] = w.num_pages
    sl[1], sl[2] = -3, bt.shape[1] * 16 + 1
    wt = weights_for(w, 119, 5)            # sequence 3 is longer than its weights
    run_evict(w, wt, budget=50, recent=5, block_table=bt, seq_lens=sl, expect=3)
    free = np.setdiff1d(np.arange(w.num_pages), w.block_table[w.block_table >= 0])
    dst = free[:18].reshape(6, 3).astype(np.int32)  # 48 tokens: too short for 50
    run_evict(w, weights_for(w, 120, 6), budget=50, dst=dst, expect=2)
    dst[5, 1] = -1
    run_evict(w, weights_for(w, 120, 7), budget=40, dst=dst, expect=1)


def _paths(g, B, q_len, n):
    path = np.full((B, n), 1 << 20, dtype=np.int32)
    acc = g.integers(0, min(n, q_len), size=B, endpoint=True).astype(np.int32)
    for b in range(B):
        path[b, :acc[b]] = np.sort(g.choice(q_len, acc[b], replace=False))
    return path, acc


def run_commit(w, path, acc, q_len, *, block_table=None, seq_lens=None, expect=0):
    bt = w.block_table if block_table is None else block_table
    sl = w.seq_lens if seq_lens is None else seq_lens
    k, v, btd, sld, pd, ad = cuda(w.k_pool.clone(), None if w.v_pool is None else w.v_pool.clone(),
                                  bt, sl, path, acc)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = zl.kv_commit(k, v, btd, sld, pd, ad, page_size=w.page_size, q_len=q_len,
                       layout=w.layout, err_flags=err)
    torch.cuda.synchronize()
    rk, rv, rnew, rerr = commit(u16(nhd(w, w.k_pool)),
                                None if w.v_pool is None else u16(nhd(w, w.v_pool)), bt, sl, path,
                                acc, page_size=w.page_size, q_len=q_len, num_pages=w.num_pages)
    assert int(err.item()) == rerr == expect
    assert np.array_equal(new.cpu().numpy(), rnew)
    assert np.array_equal(u16(nhd(w, k)), rk)
    if v is not None:
        assert np.array_equal(u16(nhd(w, v)), rv)


@pytest.mark.parametrize("q_len", [1, 2, 16, 17, 64, 128])
@pytest.mark.parametrize("layout,P", [("NHD", 16), ("HND", 48)])
def test_commit_paths(q_len, layout, P):
    w = wl.random_case(3200 + q_len, B=6, Hq=8, Hkv=2, page_size=P, layout=layout,
                       lens=[q_len, q_len + 1, 300, 200, 130, 129])
    path, acc = _paths(np.random.default_rng(q_len), 6, q_len, q_len)
    run_commit(w, path, acc, q_len)
    # unsorted, with repeats: every row is read before any is written
    g = np.random.default_rng(1)
    path = g.integers(0, q_len, size=(6, q_len)).astype(np.int32)
    run_commit(w, path, np.full(6, q_len, dtype=np.int32), q_len)


def test_commit_latent_pool_and_short_path_rows():
    w = wl.random_case(3210, B=3, Hq=128, Hkv=1, D=576, page_size=64, mla=True, D_v=512,
                       lens=[300, 64, 200])
    path, acc = _paths(np.random.default_rng(3), 3, 20, 5)
    run_commit(w, path, acc, 20)


def test_commit_errors():
    w = wl.random_case(3220, B=7, Hq=8, Hkv=2, lens=[100, 90, 80, 120, 64, 110, 95])
    q_len = 12
    path, acc = _paths(np.random.default_rng(4), 7, q_len, q_len)
    acc[:] = 3
    path[:, :3] = [2, 5, 9]
    bt, sl = w.block_table.copy(), w.seq_lens.copy()
    acc[0], acc[1] = -1, q_len + 1
    path[2, 1], path[3, 2] = -1, q_len
    sl[4] = q_len - 1
    sl[5] = bt.shape[1] * 16 + 1
    bt[6, 94 // 16] = -1
    run_commit(w, path, acc, q_len, block_table=bt, seq_lens=sl, expect=19)
    acc[:] = 6   # more than a row of the path holds
    run_commit(w, path[:, :5].copy(), acc, q_len, expect=16)


def test_decode_loop():
    """Speculative decode over a held cache: append and verify a drafted tree,
    commit its path, decode a token with weights, evict, attend again -- on one
    stream, against the same steps in the plain forms."""
    B, Hq, Hkv, q_len, P, D, budget = 3, 8, 2, 6, 16, 128, 96
    lens = np.array([100, 40, 131], dtype=np.int32)
    w = wl.random_case(3300, B=B, Hq=Hq, Hkv=Hkv, lens=[160, 160, 160], poison=False)
    g = np.random.default_rng(9)
    gt = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=gt).to(torch.bfloat16)  # noqa: E731
    k, v, bt = cuda(w.k_pool, w.v_pool, w.block_table)
    kr, vr = u16(k).copy(), u16(v).copy()
    tof = lambda x: torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    wt = torch.zeros(B, Hkv, 160, device="cuda")
    wr, wr_tol = np.zeros((B, Hkv, 160)), np.zeros((B, Hkv, 160))
    sl = torch.from_numpy(lens).cuda()
    slr = lens.copy()
    for step in range(3):
        # verify a drafted tree
        sl = sl + q_len
        slr = slr + q_len
        par = [[-1] + [int(g.integers(-1, i)) for i in range(1, q_len)] for _ in range(B)]
        mask = zl.tree_mask(par)
        q, kn, vn = rnd(B, q_len, Hq, D), rnd(B, q_len, Hkv, D), rnd(B, q_len, Hkv, D)
        out = zl.decode_attn(q.cuda(), k, v, bt, sl, page_size=P, scale=w.scale, softcap=12.0,
                             tree_mask=mask.cuda(), k_new=kn.cuda(), v_new=vn.cuda())
        for b in range(B):
            for i in range(q_len):
                t = slr[b] - q_len + i
                kr[w.block_table[b, t // P], t % P] = u16(kn)[b, i]
                vr[w.block_table[b, t // P], t % P] = u16(vn)[b, i]
        ref = attention(f64(q), f64(tof(kr)), f64(tof(vr)), w.block_table, slr, scale=w.scale,
                        softcap=12.0, mask=mask)
        check(f64(out), ref.out, ref.out_tol, f"tree {step}")
        # commit the accepted path
        path, acc = _paths(g, B, q_len, q_len)
        sl = zl.kv_commit(k, v, bt, sl, *cuda(path, acc), page_size=P, q_len=q_len)
        kr, vr, slr, _ = commit(kr, vr, w.block_table, slr, path, acc, page_size=P, q_len=q_len,
                                num_pages=w.num_pages)
        # one token with weights
        sl, slr = sl + 1, slr + 1
        q, kn, vn = rnd(B, 1, Hq, D), rnd(B, 1, Hkv, D), rnd(B, 1, Hkv, D)
        out = zl.decode_attn(q.cuda(), k, v, bt, sl, page_size=P, scale=w.scale, weights=wt,
                             weights_decay=0.9, k_new=kn.cuda(), v_new=vn.cuda())
        for b in range(B):
            t = slr[b] - 1
            kr[w.block_table[b, t // P], t % P] = u16(kn)[b, 0]
            vr[w.block_table[b, t // P], t % P] = u16(vn)[b, 0]
        ref = attention(f64(q), f64(tof(kr)), f64(tof(vr)), w.block_table, slr, scale=w.scale,
                        tokens=160, decay=0.9, old=f64(wt.clone().fill_(0)))
        check(f64(out), ref.out, ref.out_tol, f"token {step}")
        inside = np.arange(160)[None, None] < slr[:, None, None]
        wr = np.where(inside, 0.9 * wr, wr) + ref.weights
        wr_tol = wr_tol + ref.weights_tol + 2.0 ** -22 * np.abs(wr)
        check(f64(wt), wr, wr_tol, f"weights {step}")
        # back to the budget; the plain form takes the GPU's weights (their order decides)
        before = wt.cpu().numpy()
        sl, kept = zl.kv_evict(k, v, bt, sl, wt, page_size=P, budget=budget, sink=2, recent=30)
        kr, vr, wn, keptr, slr, _ = evict(kr, vr, before, w.block_table, slr, page_size=P,
                                          budget=budget, sink=2, recent=30, num_pages=w.num_pages)
        assert np.array_equal(kept.cpu().numpy(), keptr)
        assert np.array_equal(wt.cpu().numpy(), wn)
        moved, moved_tol = wr.copy(), wr_tol.copy()
        for b in range(B):
            for h in range(Hkv):
                idx = keptr[b, h][keptr[b, h] >= 0]
                moved[b, h, :len(idx)] = wr[b, h, idx]
                moved_tol[b, h, :len(idx)] = wr_tol[b, h, idx]
        wr, wr_tol = moved, moved_tol
        assert np.array_equal(u16(k), kr) and np.array_equal(u16(v), vr)
        assert np.array_equal(sl.cpu().numpy(), slr)


def test_evict_and_commit_in_a_graph():
    w = wl.random_case(3310, B=4, Hq=8, Hkv=2, lens=[300, 200, 100, 90])
    wt = weights_for(w, 300, 8)
    path, acc = _paths(np.random.default_rng(5), 4, 10, 10)
    k0, v0, bt, sl, wd, pd, ad = cuda(w.k_pool, w.v_pool, w.block_table, w.seq_lens, wt, path, acc)

    def step(k, v, wts):
        mid = zl.kv_commit(k, v, bt, sl, pd, ad, page_size=16, q_len=10)
        return zl.kv_evict(k, v, bt, mid, wts, page_size=16, budget=80, sink=1, recent=9)

    ke, ve, we = k0.clone(), v0.clone(), wd.clone()
    new_e, kept_e = step(ke, ve, we)
    k, v, wg = k0.clone(), v0.clone(), wd.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new, kept = step(k, v, wg)
    for _ in range(3):
        k.copy_(k0), v.copy_(v0), wg.copy_(wd)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(new, new_e) and torch.equal(kept, kept_e)
    assert torch.equal(k.view(torch.int16), ke.view(torch.int16))
    assert torch.equal(v.view(torch.int16), ve.view(torch.int16))
    assert torch.equal(wg, we)
