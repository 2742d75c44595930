"""A cached token's sum of weights stays its own through the decode loop: what
the operators that move tokens leave behind the new length is no new token's
start. The references carry the sums by token, not by position."""
import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from paged_decode_attention_gqa_gb300 import workloads as wl
from plain_ops import attention, check, commit, evict, f64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def u16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def as_f64(x):
    return torch.from_numpy(x.view(np.int16)).view(BF16).double().numpy()


class Sums:
    """Sums of weights by token: the cache of every (sequence, kv head) is a list
    of tokens in the order of their positions."""

    def __init__(self, B, Hkv, lens):
        self.B, self.H, self.n = B, Hkv, 0
        self.val, self.tol = {}, {}
        self.cache = [[[self.new() for _ in range(int(lens[b]))] for _ in range(Hkv)]
                      for b in range(B)]

    def new(self):
        self.n += 1
        self.val[self.n] = self.tol[self.n] = 0.0
        return self.n

    def append(self, n):
        for b in range(self.B):
            for h in range(self.H):
                self.cache[b][h] += [self.new() for _ in range(n)]

    def add(self, w, tol, decay):
        """w, tol [B, Hkv, T]: one call's weights by position."""
        for b in range(self.B):
            for h in range(self.H):
                for t, tok in enumerate(self.cache[b][h]):
                    v = decay * self.val[tok] + w[b, h, t]
                    # the old sum's error, this call's, and the fma's rounding
                    self.tol[tok] = decay * self.tol[tok] + tol[b, h, t] + 2.0 ** -22 * abs(v)
                    self.val[tok] = v

    def keep(self, b, h, positions):
        self.cache[b][h] = [self.cache[b][h][int(t)] for t in positions]

    def rows(self, T):
        """By position, zeros behind the length."""
        v, tol = np.zeros((self.B, self.H, T)), np.zeros((self.B, self.H, T))
        for b in range(self.B):
            for h in range(self.H):
                for t, tok in enumerate(self.cache[b][h]):
                    v[b, h, t], tol[b, h, t] = self.val[tok], self.tol[tok]
        return v, tol


@pytest.mark.parametrize("swap", [False, True])
def test_decode_and_evict_loop(swap):
    """A token per step, its weights, then back to the budget. swap: the kept sums
    go to the other of two buffers each time."""
    B, Hq, Hkv, P, D, T, budget, steps = 2, 8, 2, 16, 128, 80, 48, 30
    lens = np.array([44, 48], dtype=np.int32)
    w = wl.random_case(3400, B=B, Hq=Hq, Hkv=Hkv, lens=[T, T], poison=False)
    gt = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=gt).to(BF16)  # noqa: E731
    k, v, bt = w.k_pool.cuda(), w.v_pool.cuda(), torch.from_numpy(w.block_table).cuda()
    kr, vr = u16(k).copy(), u16(v).copy()
    bufs = [torch.zeros(B, Hkv, T, device="cuda") for _ in range(2)]
    if swap:
        bufs[1].fill_(7.0)  # what an earlier use of the buffer left
    sums = Sums(B, Hkv, lens)
    sl, slr = torch.from_numpy(lens).cuda(), lens.copy()
    for step in range(steps):
        wt = bufs[step % 2 if swap else 0]
        sl, slr = sl + 1, slr + 1
        sums.append(1)
        q, kn, vn = rnd(B, 1, Hq, D), rnd(B, 1, Hkv, D), rnd(B, 1, Hkv, D)
        zl.decode_attn(q.cuda(), k, v, bt, sl, page_size=P, scale=w.scale, weights=wt,
                       weights_decay=0.9, k_new=kn.cuda(), v_new=vn.cuda())
        for b in range(B):
            t = slr[b] - 1
            kr[w.block_table[b, t // P], t % P] = u16(kn)[b, 0]
            vr[w.block_table[b, t // P], t % P] = u16(vn)[b, 0]
        ref = attention(f64(q), as_f64(kr), as_f64(vr), w.block_table, slr, scale=w.scale,
                        tokens=T)
        sums.add(ref.weights, ref.weights_tol, 0.9)
        check(f64(wt), *sums.rows(T), f"weights {step}")
        before = wt.cpu().numpy()
        out = bufs[(step + 1) % 2] if swap else None
        sl, kept = zl.kv_evict(k, v, bt, sl, wt, page_size=P, budget=budget, sink=2, recent=6,
                               weights_out=out, clear_weights=True)
        kr, vr, _, keptr, slr, _ = evict(kr, vr, before, w.block_table, slr, page_size=P,
                                         budget=budget, sink=2, recent=6, num_pages=w.num_pages)
        assert np.array_equal(kept.cpu().numpy(), keptr)
        for b in range(B):
            for h in range(Hkv):
                sums.keep(b, h, keptr[b, h][keptr[b, h] >= 0])
        check(f64(wt if out is None else out), *sums.rows(T), f"kept weights {step}")


def run_clear(w, wt, *, out_tokens=None, dst=None, **kw):
    """kv_evict with clear_weights against the plain form, whose rows are then
    cleared behind the new length."""
    k, v = w.k_pool.cuda(), w.v_pool.cuda()
    bt, sl = torch.from_numpy(w.block_table).cuda(), torch.from_numpy(w.seq_lens).cuda()
    wd = wt.cuda()
    out = None if out_tokens is None else torch.full((w.B, w.Hkv, out_tokens), 5.0)
    od = None if out is None else out.cuda()
    new, kept = zl.kv_evict(k, v, bt, sl, wd, page_size=w.page_size, clear_weights=True,
                            weights_out=od, dst_block_table=None if dst is None
                            else torch.from_numpy(dst).cuda(), **kw)
    kr, vr, wr, keptr, newr, _ = evict(
        u16(w.k_pool), u16(w.v_pool), wt.numpy(), w.block_table, w.seq_lens,
        page_size=w.page_size, num_pages=w.num_pages, dst_table=dst,
        weights_out=None if out is None else out.numpy(), sink=kw.get("sink", 0),
        recent=kw.get("recent", 0), budget=kw["budget"])
    for b in range(w.B):
        wr[b, :, newr[b]:w.seq_lens[b] if out is None else out_tokens] = 0
    assert np.array_equal(kept.cpu().numpy(), keptr)
    assert np.array_equal(new.cpu().numpy(), newr)
    assert np.array_equal((wd if od is None else od).cpu().numpy(), wr)
    if od is not None:
        assert torch.equal(wd.cpu(), wt)
    assert np.array_equal(u16(k), kr) and np.array_equal(u16(v), vr)


@pytest.mark.parametrize("out_tokens", [None, 64, 320])
@pytest.mark.parametrize("budget,sink,recent", [(64, 0, 0), (64, 4, 16), (50, 7, 43), (1, 0, 0),
                                                (33, 0, 33), (33, 33, 0), (60, 0, 60),
                                                (299, 1, 2)])
def test_clear_behind_the_new_length(out_tokens, budget, sink, recent):
    if out_tokens == 64 and budget > 64:
        pytest.skip("the rows would not hold the budget")
    w = wl.random_case(3410, B=6, Hq=8, Hkv=2, lens=[300, 1, 0, 64, 65, 150])
    wt = torch.rand(6, 2, 310, generator=torch.Generator().manual_seed(budget)) + 0.5
    run_clear(w, wt, out_tokens=out_tokens, budget=budget, sink=sink, recent=recent)


@pytest.mark.parametrize("L,T,budget,recent", [(20000, 20000, 9001, 8000), (20000, 20011, 500, 0),
                                               (131073, 131080, 4097, 1000)])
def test_clear_long_rows(L, T, budget, recent):
    """Rows over a cluster of CTAs, and rows that no cluster holds."""
    w = wl.random_case(3420, B=2, Hq=1, Hkv=1, page_size=128, lens=[L, 40], poison=False,
                       pool_factor=3.0)
    wt = torch.rand(2, 1, T, generator=torch.Generator().manual_seed(L)) + 0.5
    run_clear(w, wt, budget=budget, sink=3, recent=recent)
    run_clear(w, wt, budget=budget, sink=3, recent=recent, out_tokens=T)
    free = np.setdiff1d(np.arange(w.num_pages), w.block_table[w.block_table >= 0])
    n = (budget + 127) // 128
    run_clear(w, wt, budget=budget, recent=recent, dst=free[:2 * n].reshape(2, n).astype(np.int32))


@pytest.mark.parametrize("clear", [False, True])
def test_evict_by_a_view_of_wider_rows(clear):
    """weights[:, :, :n] of wide rows: the result of rows of n, nothing past n touched."""
    w = wl.random_case(3425, B=3, Hq=8, Hkv=2, lens=[300, 120, 33])
    wt = torch.rand(3, 2, 301, generator=torch.Generator().manual_seed(4)) + 0.5
    got = []
    for width in (301, 5000):
        k, v = w.k_pool.cuda(), w.v_pool.cuda()
        big = torch.full((3, 2, width), 9.0, device="cuda")
        big[:, :, :301] = wt.cuda()
        new, kept = zl.kv_evict(k, v, torch.from_numpy(w.block_table).cuda(),
                                torch.from_numpy(w.seq_lens).cuda(), big[:, :, :301],
                                page_size=16, budget=100, sink=2, recent=9, clear_weights=clear)
        got.append((new, kept, k.view(torch.int16), v.view(torch.int16),
                    big[:, :, :301].contiguous()))
        assert bool((big[:, :, 301:] == 9.0).all())
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_clear_leaves_bad_sequences_alone():
    w = wl.random_case(3430, B=3, Hq=8, Hkv=2, lens=[100, 90, 80])
    sl = torch.tensor([-1, 101, 80], dtype=torch.int32).cuda()
    wt = torch.rand(3, 2, 100, generator=torch.Generator().manual_seed(1)) + 0.5
    wd = wt.cuda()
    zl.kv_evict(w.k_pool.cuda(), w.v_pool.cuda(), torch.from_numpy(w.block_table).cuda(), sl, wd,
                page_size=16, budget=32, clear_weights=True)
    assert torch.equal(wd[:2].cpu(), wt[:2])
    assert not wd[2, :, 32:80].any() and torch.equal(wd[2, :, 80:].cpu(), wt[2, :, 80:])


def test_evict_struct_without_the_last_field():
    """A caller built before weights_clear was there: nothing is cleared."""
    w = wl.random_case(3440, B=1, Hq=2, Hkv=1, lens=[40])
    k, v, bt, sl = (x.cuda() for x in (w.k_pool, w.v_pool, torch.from_numpy(w.block_table),
                                       torch.from_numpy(w.seq_lens)))
    wt = torch.ones(1, 1, 40, device="cuda")
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.zeros(1, 1, 8, dtype=torch.int32, device="cuda")
    p = zl.EvictParams()
    p.struct_size = zl.EvictParams.weights_clear.offset
    p.k_pool, p.v_pool = k.data_ptr(), v.data_ptr()
    p.page_stride, p.token_stride, p.head_stride = k.stride(0), k.stride(1), k.stride(2)
    p.block_table, p.block_table_stride, p.seq_lens = bt.data_ptr(), bt.shape[1], sl.data_ptr()
    p.new_lens, p.kept, p.weights = new.data_ptr(), kept.data_ptr(), wt.data_ptr()
    p.weights_tokens = p.weights_seq_stride = p.weights_head_stride = 40
    p.B, p.Hkv, p.D_k, p.D_v, p.page_size, p.num_pages = 1, 1, 128, 128, 16, w.num_pages
    p.budget, p.recent, p.weights_clear = 8, 8, 1  # the last lies outside the given size
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert zl.lib().zl_kv_evict(ctypes.byref(p), stream) == zl.OK
    torch.cuda.synchronize()
    assert new.tolist() == [8] and kept.tolist() == [[list(range(32, 40))]]
    assert bool((wt == 1).all())


def run_commit(w, path, acc, q_len, wt, *, seq_lens=None, block_table=None):
    """kv_commit with weights: the plain form for the pools, sums by hand."""
    bt = w.block_table if block_table is None else block_table
    sl = w.seq_lens if seq_lens is None else seq_lens
    k, v = w.k_pool.cuda(), w.v_pool.cuda()
    big = torch.full((w.B, w.Hkv + 1, wt.shape[2] + 9), 3.0, device="cuda")
    view = big[:, :w.Hkv, 5:5 + wt.shape[2]]  # rows inside a larger buffer
    view.copy_(wt)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = zl.kv_commit(k, v, torch.from_numpy(bt).cuda(), torch.from_numpy(sl).cuda(),
                       torch.from_numpy(path).cuda(), torch.from_numpy(acc).cuda(),
                       page_size=w.page_size, q_len=q_len, weights=view, err_flags=err)
    long = sl > wt.shape[2]
    slr = np.where(long, -1, sl).astype(np.int32)  # a bad length for the plain form
    kr, vr, newr, errr = commit(u16(w.k_pool), u16(w.v_pool), bt, slr, path, acc,
                                page_size=w.page_size, q_len=q_len, num_pages=w.num_pages)
    newr = np.where(long, sl, newr)
    want = wt.numpy().copy()
    for b in range(w.B):
        ctx, n = int(sl[b]) - q_len, int(newr[b]) - int(sl[b]) + q_len
        if newr[b] == sl[b] and (slr[b] < q_len or n != acc[b]):
            continue  # refused: nothing moves
        want[b, :, ctx:ctx + n] = wt.numpy()[b][:, ctx + path[b, :n]]
        want[b, :, ctx + n:sl[b]] = 0
    assert int(err.item()) == errr
    assert np.array_equal(new.cpu().numpy(), newr)
    assert np.array_equal(view.cpu().numpy(), want)
    big[:, :w.Hkv, 5:5 + wt.shape[2]] = 3.0
    assert bool((big == 3.0).all())
    assert np.array_equal(u16(k), kr) and np.array_equal(u16(v), vr)
    return errr


@pytest.mark.parametrize("q_len", [1, 2, 16, 17, 64, 128])
def test_commit_moves_the_sums(q_len):
    w = wl.random_case(3450 + q_len, B=6, Hq=8, Hkv=2, poison=False,
                       lens=[q_len, q_len + 1, 300, 200, 130, 129])
    wt = torch.rand(6, 2, 301, generator=torch.Generator().manual_seed(q_len)) + 0.5
    g = np.random.default_rng(q_len)
    path = g.integers(0, q_len, size=(6, q_len)).astype(np.int32)  # unsorted, with repeats
    acc = g.integers(0, q_len, size=6, endpoint=True).astype(np.int32)
    acc[0], acc[1] = q_len, 0
    assert run_commit(w, path, acc, q_len, wt) == 0


def test_commit_of_bad_sequences_leaves_their_sums():
    w = wl.random_case(3460, B=6, Hq=8, Hkv=2, lens=[100, 90, 80, 120, 64, 110], poison=False)
    path = np.tile(np.array([2, 5, 9], dtype=np.int32), (6, 1))
    acc = np.array([3, -1, 3, 3, 3, 2], dtype=np.int32)
    path[2, 1] = 12
    sl, bt = w.seq_lens.copy(), w.block_table.copy()
    sl[4] = 11
    bt[5, 109 // 16] = -1                    # a row that does not move; its sum does
    wt = torch.rand(6, 2, 115, generator=torch.Generator().manual_seed(2)) + 0.5
    assert run_commit(w, path, acc, 12, wt, seq_lens=sl, block_table=bt) == 2 + 16 + 1


def test_verify_commit_and_evict_loop():
    """Drafted trees verified with weights, their paths committed, the cache back to
    the budget: every token keeps its own sum."""
    B, Hq, Hkv, q_len, P, D, T, budget = 2, 8, 2, 7, 16, 128, 80, 48
    lens = np.array([44, 48], dtype=np.int32)
    w = wl.random_case(3470, B=B, Hq=Hq, Hkv=Hkv, lens=[T, T], poison=False)
    g, gt = np.random.default_rng(6), torch.Generator().manual_seed(12)
    rnd = lambda *s: torch.randn(*s, generator=gt).to(BF16)  # noqa: E731
    k, v, bt = w.k_pool.cuda(), w.v_pool.cuda(), torch.from_numpy(w.block_table).cuda()
    kr, vr = u16(k).copy(), u16(v).copy()
    wt = torch.zeros(B, Hkv, T, device="cuda")
    sums = Sums(B, Hkv, lens)
    sl, slr = torch.from_numpy(lens).cuda(), lens.copy()
    for step in range(8):
        sl, slr = sl + q_len, slr + q_len
        sums.append(q_len)
        mask = zl.tree_mask([[-1] + [int(g.integers(-1, i)) for i in range(1, q_len)]
                             for _ in range(B)])
        q, kn, vn = rnd(B, q_len, Hq, D), rnd(B, q_len, Hkv, D), rnd(B, q_len, Hkv, D)
        zl.decode_attn(q.cuda(), k, v, bt, sl, page_size=P, scale=w.scale, weights=wt,
                       tree_mask=mask.cuda(), k_new=kn.cuda(), v_new=vn.cuda())
        for b in range(B):
            for i in range(q_len):
                t = slr[b] - q_len + i
                kr[w.block_table[b, t // P], t % P] = u16(kn)[b, i]
                vr[w.block_table[b, t // P], t % P] = u16(vn)[b, i]
        ref = attention(f64(q), as_f64(kr), as_f64(vr), w.block_table, slr, scale=w.scale,
                        mask=mask, tokens=T)
        sums.add(ref.weights, ref.weights_tol + q_len * 4 * 2.0 ** -22 * ref.weights, 1.0)
        acc = g.integers(0, q_len, size=B, endpoint=True).astype(np.int32)
        path = np.zeros((B, q_len), dtype=np.int32)
        for b in range(B):
            path[b, :acc[b]] = np.sort(g.choice(q_len, acc[b], replace=False))
        sl = zl.kv_commit(k, v, bt, sl, torch.from_numpy(path).cuda(), torch.from_numpy(acc).cuda(),
                          page_size=P, q_len=q_len, weights=wt)
        kr, vr, newr, _ = commit(kr, vr, w.block_table, slr, path, acc, page_size=P, q_len=q_len,
                                 num_pages=w.num_pages)
        for b in range(B):
            ctx = int(slr[b]) - q_len
            for h in range(Hkv):
                sums.keep(b, h, list(range(ctx)) + [ctx + int(x) for x in path[b, :acc[b]]])
        slr = newr
        check(f64(wt), *sums.rows(T), f"committed weights {step}")
        before = wt.cpu().numpy()
        sl, kept = zl.kv_evict(k, v, bt, sl, wt, page_size=P, budget=budget, sink=2, recent=6,
                               clear_weights=True)
        kr, vr, _, keptr, slr, _ = evict(kr, vr, before, w.block_table, slr, page_size=P,
                                         budget=budget, sink=2, recent=6, num_pages=w.num_pages)
        assert np.array_equal(kept.cpu().numpy(), keptr)
        for b in range(B):
            for h in range(Hkv):
                sums.keep(b, h, keptr[b, h][keptr[b, h] >= 0])
        check(f64(wt), *sums.rows(T), f"kept weights {step}")
        assert np.array_equal(sl.cpu().numpy(), slr)
