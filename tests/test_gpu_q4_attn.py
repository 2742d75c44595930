"""Decode attention over a 4-bit cache against the definition in 64 bits over the values
that the cache holds (tolerances: plain_q4.tolerance)."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_q4 import ROW, Cache, attention, bf16, pack, random_rows

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def queries(c, q_len, Hq, size=1.0):
    q = c.g.standard_normal((len(c.lens), q_len, Hq, 128)) * size
    return torch.from_numpy(q).to(torch.bfloat16)


def run(c, q, **kw):
    pool, bt, sl = c.on_gpu()
    lse = torch.full(q.shape[:3], 77.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = zl.decode_attn_q4(q.cuda(), pool, bt, sl, page_size=c.P, scale=SCALE, lse=lse,
                            layout=c.layout, err_flags=err, **kw)
    return bf16(out), bf16(lse), int(err.item())


def check(c, q, **kw):
    out, lse, err = run(c, q, **kw)
    assert err == 0
    want, want_lse, t_out, t_lse = attention(bf16(q), [c.kv(b) for b in range(len(c.lens))],
                                             c.lens, SCALE)
    assert np.isfinite(out).all()
    worst = (np.abs(out - want) - t_out).max()
    assert worst <= 0, worst
    none = np.isinf(want_lse)
    assert (lse[none] == -np.inf).all() and (out[none] == 0).all()
    assert (np.abs(lse[~none] - want_lse[~none]) <= t_lse[~none]).all()
    return out, lse


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("lens,Hq,Hkv,P", [
    ([1], 1, 1, 16), ([16], 4, 2, 16), ([17, 15, 1, 33], 8, 2, 16), ([0, 5, 0, 64], 8, 8, 32),
    ([100, 900], 32, 8, 16), ([255, 256, 257], 12, 6, 48), ([700], 5, 1, 64),
    ([300, 1], 64, 4, 16), ([513], 32, 1, 128), ([80] * 40, 10, 5, 16), ([77, 500], 128, 1, 16),
    ([333, 20], 21, 7, 16),
])
def test_shapes(lens, Hq, Hkv, P, layout):
    c = Cache(sum(lens) + Hq, lens, Hkv, P, layout)
    q = queries(c, 1, Hq, 2.0)
    a = check(c, q)
    b = check(c, q, max_seq_len=max(lens))
    again = run(c, q)
    assert np.array_equal(a[0], again[0]) and np.array_equal(a[1], again[1])
    del b


@pytest.mark.parametrize("q_len,Hq,Hkv,lens", [
    (2, 8, 2, [2, 17, 300]), (3, 8, 2, [1, 2, 3, 100]), (4, 32, 8, [600, 4, 33]),
    (5, 16, 16, [50, 5, 16]), (17, 4, 2, [17, 40, 3]), (128, 3, 1, [128, 500, 100]),
    (7, 40, 2, [7, 90]), (16, 16, 4, [15, 16, 129]),
])
def test_several_query_tokens(q_len, Hq, Hkv, lens):
    c = Cache(q_len * 31 + Hq, lens, Hkv)
    q = queries(c, q_len, Hq)
    check(c, q)
    check(c, q, num_ctas=5)


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 16, 100, 500])
def test_any_number_of_ctas(num_ctas):
    c = Cache(3, [1000, 1, 0, 350, 64], 4, 16)
    check(c, queries(c, 1, 16, 2.0), num_ctas=num_ctas)
    check(c, queries(c, 5, 16, 2.0), num_ctas=num_ctas)


def test_large_calls_put_heads_side_by_side():
    for Hkv, layout in ((8, "NHD"), (6, "HND"), (7, "NHD"), (3, "NHD"), (16, "NHD")):
        c = Cache(40 + Hkv, [700, 333, 17, 0, 150], Hkv, 32, layout)
        q = queries(c, 1, Hkv * 2, 2.0)
        check(c, q, max_seq_len=200000)
        check(c, q, max_seq_len=200000, num_ctas=11)


@pytest.mark.parametrize("B,hi,q_len,Hq,Hkv", [(51, 32, 5, 32, 8), (64, 120, 1, 32, 8),
                                               (40, 90, 1, 12, 6), (90, 60, 2, 8, 4)])
@pytest.mark.parametrize("bound", [False, True])
def test_many_short_sequences(B, hi, q_len, Hq, Hkv, bound):
    """More heads than CTAs, each of a few tiles."""
    lens = [q_len + (i * 37) % (hi - q_len + 1) for i in range(B - 2)] + [hi, 0]
    c = Cache(33, lens, Hkv)
    check(c, queries(c, q_len, Hq), max_seq_len=hi if bound else 0)


CLUSTERS = [([700, 0, 33, 1999], 8, 2, 1, 16), ([2000, 1, 513, 257], 32, 8, 1, 48),
            ([900], 2, 2, 1, 16), ([1500, 40], 5, 1, 3, 32), ([4000], 32, 1, 2, 64),
            ([300, 600, 1200, 2400, 5], 16, 4, 1, 16), ([1000] * 19, 8, 1, 2, 16),
            ([7000, 300], 8, 1, 1, 128)]


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("lens,Hq,Hkv,q_len,P", CLUSTERS)
def test_few_units_with_a_bound(lens, Hq, Hkv, q_len, P, layout):
    """Several CTAs to a unit, which merge it themselves where the bound is short."""
    c = Cache(34, [L if L == 0 else max(L, q_len) for L in lens], Hkv, P=P, layout=layout)
    check(c, queries(c, q_len, Hq), max_seq_len=max(lens))


def test_few_units_with_a_bound_that_does_not_hold():
    c = Cache(36, [2500, 40, 1100], 2)
    for bound in (1000, 700):
        check(c, queries(c, 1, 8), max_seq_len=bound)


def test_few_units_with_a_bound_and_bad_pages_numbers_and_lengths():
    """A bad page, a NaN block and a bad length reach the rows that they reach without one."""
    c = Cache(35, [1400, 900, 700, 64], 2)
    q = queries(c, 2, 8)
    q[1, 0, 3, 9] = float("nan")
    c.bt[0, 50] = -1  # tokens 800 .. 815 of sequence 0
    page, slot = c.place(2, 300)
    c.pool[page, slot, 1, 136 + 2] = 255
    c.lens[3] = 10 ** 6
    a = run(c, q, num_ctas=5)
    b = run(c, q, max_seq_len=1400)
    assert a[2] == b[2] == zl.DEVERR_BAD_PAGE | zl.DEVERR_BAD_SEQ_LEN
    for x, y in zip(a[:2], b[:2]):
        assert np.array_equal(np.isnan(x), np.isnan(y)) and np.array_equal(np.isinf(x), np.isinf(y))
        ok = np.isfinite(x)
        # both are within a bf16 rounding and 2^-10 (P) of the same sums
        assert np.allclose(x[ok], y[ok], rtol=2.0 ** -7, atol=2.0 ** -9)
    assert not b[0][[0, 3]].any() and np.isnan(b[0][1, 0, 3]).all()
    assert np.isnan(b[0][2, :, 4:, 32:48]).all() and np.isfinite(b[0][2, :, :4]).all()


def test_remapped_pages_give_the_same_bits():
    c = Cache(21, [400, 90], 2)
    q = queries(c, 1, 8)
    out, lse, _ = run(c, q)
    old = [c.rows(b, np.arange(L)).copy() for b, L in enumerate(c.lens)]
    perm = np.roll(np.arange(c.pages), 5).astype(np.int32)
    c.bt = np.where(c.bt >= 0, perm[c.bt.clip(min=0)], -1).astype(np.int32)
    for b, L in enumerate(c.lens):
        c.put(b, np.arange(L), old[b])
    out2, lse2, _ = run(c, q)
    assert np.array_equal(out, out2) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e30])
def test_queries_of_any_size(size):
    """Far outside fp16's range: the row's factor carries it. (Scores of 1e30 are within
    32 bits; the softmax picks single tokens.)"""
    c = Cache(22, [70, 33], 2, spread=0.5)
    q = queries(c, 2, 8).double()
    q = (q * size * torch.exp(torch.randn(2, 2, 8, 1, dtype=torch.float64,
                                          generator=torch.Generator().manual_seed(1)))).bfloat16()
    out, lse, err = run(c, q)
    want, want_lse, t_out, t_lse = attention(bf16(q), [c.kv(b) for b in range(2)], c.lens, SCALE)
    assert err == 0 and (np.abs(out - want) <= t_out).all()
    assert (np.abs(lse - want_lse) <= t_lse).all()


def test_scores_that_grow_along_the_context():
    """The softmax base moves again and again, and late tokens outweigh early ones; and
    the other way round."""
    for turn in (1, -1):
        c = Cache(23, [600], 1, fill=False)
        k = np.linspace(0, 4, 600)[::turn, None, None] * np.ones((600, 1, 128))
        v = bf16(random_rows(c.g, 600, 1))
        c.put(0, np.arange(600), pack(k, v))
        q = torch.ones(1, 1, 8, 128, dtype=torch.bfloat16) * torch.arange(1, 9)[None, None, :, None]
        check(c, q.to(torch.bfloat16))
        check(c, -q.to(torch.bfloat16))


def test_a_single_heavy_token_and_equal_tokens():
    c = Cache(24, [500], 2, fill=False)
    k = np.zeros((500, 2, 128))
    k[123, 0] = 6.0
    v = bf16(random_rows(c.g, 500, 2))
    c.put(0, np.arange(500), pack(k, v))
    check(c, torch.full((1, 1, 4, 128), 3.0, dtype=torch.bfloat16))


def test_bad_pages_zero_the_rows_that_reach_them():
    c = Cache(25, [100, 64, 40], 2)
    q = queries(c, 3, 4)
    good, good_lse, _ = run(c, q)
    c.bt[0, 6] = c.pages + 5      # tokens 96 .. 99: every query token of sequence 0
    c.bt[2, 1] = -7               # 16 .. 31
    out, lse, err = run(c, q)
    assert err == zl.DEVERR_BAD_PAGE
    assert not out[[0, 2]].any() and (lse[[0, 2]] == -np.inf).all()
    assert np.array_equal(out[1], good[1]) and np.array_equal(lse[1], good_lse[1])
    # a bad page with the newest token only: the two tokens before it keep their rows
    c = Cache(26, [97, 50], 2)
    q = queries(c, 3, 4)
    good, good_lse, _ = run(c, q)
    c.bt[0, 6] = -1
    out, lse, err = run(c, q)
    assert err == zl.DEVERR_BAD_PAGE and not out[0, 2].any()
    for x, y in ((out, good), (lse, good_lse)):
        assert np.allclose(x[0, :2], y[0, :2], rtol=2 ** -7, atol=1e-3)
        assert np.array_equal(x[1], y[1])


def test_bad_lengths():
    c = Cache(27, [30, 20, 10], 2)
    q = queries(c, 1, 4)
    good, _, _ = run(c, q)
    c.lens = [-1, 20, 10 ** 6]
    out, lse, err = run(c, q)
    assert err == zl.DEVERR_BAD_SEQ_LEN
    assert not out[[0, 2]].any() and (lse[[0, 2]] == -np.inf).all()
    assert np.array_equal(out[1], good[1])


@pytest.mark.parametrize("num_ctas", [0, 7])
def test_numbers_that_are_none(num_ctas):
    """A NaN or an infinity in a query row makes that row NaN, a NaN block of the cache
    what sees it; nothing else changes."""
    c = Cache(28, [200, 40], 2)
    q = queries(c, 1, 8)
    good, good_lse, _ = run(c, q, num_ctas=num_ctas)
    q2 = q.clone()
    q2[0, 0, 1, 5], q2[0, 0, 6, 127], q2[1, 0, 3, 0] = float("nan"), float("inf"), -float("inf")
    out, lse, err = run(c, q2, num_ctas=num_ctas)
    assert err == 0
    bad = np.zeros((2, 1, 8), bool)
    bad[0, 0, [1, 6]] = bad[1, 0, 3] = True
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    assert np.array_equal(out[~bad], good[~bad]) and np.array_equal(lse[~bad], good_lse[~bad])
    # a V block, then a K block, of sequence 0, head 1 (query heads 4 .. 7)
    page, slot = c.place(0, 150)
    c.pool[page, slot, 1, 136 + 3] = 255
    out, lse, _ = run(c, q, num_ctas=num_ctas)
    assert np.isnan(out[0, 0, 4:, 48:64]).all() and np.array_equal(lse, good_lse)
    keep = np.ones(out.shape, bool)
    keep[0, 0, 4:, 48:64] = False
    assert np.array_equal(out[keep], good[keep])
    c.pool[page, slot, 1, 128] = 255
    out, lse, _ = run(c, q, num_ctas=num_ctas)
    assert np.isnan(out[0, 0, 4:]).all() and np.isnan(lse[0, 0, 4:]).all()
    assert np.array_equal(out[0, 0, :4], good[0, 0, :4]) and np.array_equal(out[1], good[1])


@pytest.mark.parametrize("num_ctas", [0, 3])
@pytest.mark.parametrize("at", [0, 1, 2, 4])  # the drafted token with the block, from the newest
@pytest.mark.parametrize("q_len,Hq", [(5, 2), (5, 6), (7, 2)])
def test_a_nan_block_reaches_only_rows_that_see_it(q_len, Hq, at, num_ctas):
    """K or V of a drafted token without a number: the tokens before it keep their bits."""
    lens = [33, 47, 64, 300, 6]
    c = Cache(31, lens, 2)
    q = queries(c, q_len, Hq)
    good, good_lse, _ = run(c, q, num_ctas=num_ctas)
    g = Hq // 2
    for kind in ("v", "k"):
        pool = c.pool.copy()
        for b, L in enumerate(lens):
            page, slot = c.place(b, L - 1 - at)
            c.pool[page, slot, 1, (136 if kind == "v" else 128) + 3] = 255
        out, lse, err = run(c, q, num_ctas=num_ctas)
        c.pool = pool
        assert err == 0
        bad = np.zeros(out.shape, bool)
        bad[:, q_len - 1 - at:, g:, 48:64] = True
        if kind == "k":
            bad[:, q_len - 1 - at:, g:] = True
            assert np.isnan(lse[:, q_len - 1 - at:, g:]).all()
            lse[:, q_len - 1 - at:, g:] = good_lse[:, q_len - 1 - at:, g:]
        assert np.isnan(out[bad]).all()
        assert np.array_equal(out[~bad], good[~bad]) and np.array_equal(lse, good_lse)


def test_bytes_behind_the_sequence_do_not_matter():
    c = Cache(29, [37, 18], 3)
    q = queries(c, 2, 6)
    a = run(c, q)
    for b, L in enumerate(c.lens):  # NaN scales and all codes behind the last token
        end = (L + 15) // 16 * 16
        c.put(b, np.arange(L, end), np.full((end - L, 3, ROW), 255, np.uint8))
    b = run(c, q)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_far_pages_and_odd_strides():
    P, Hkv = 16, 2
    far = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
    c = Cache(30, [60], Hkv, spare=0)
    step = (5 << 30) // 4 // 16 * 16
    # rows 160 bytes apart, heads 16 rows and some bytes
    pool = far.as_strided((4, P, Hkv, ROW), (step, 160, 16 * 160 + 48, 1))
    pool.copy_(torch.from_numpy(c.pool))
    q = queries(c, 1, 4)
    _, bt, sl = c.on_gpu()
    out = zl.decode_attn_q4(q.cuda(), pool, bt, sl, page_size=P, scale=SCALE)
    want, _, _ = run(c, q)
    assert np.array_equal(bf16(out), want)


def test_long_context():
    """100000 tokens; the reference by torch in 64 bits on the GPU."""
    L, Hkv, Hq, P = 100003, 2, 8, 64
    g = torch.Generator().manual_seed(5)
    k = torch.randn(1, L, Hkv, 128, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(1, L, Hkv, 128, generator=g).to(torch.bfloat16).cuda()
    pages = -(-L // P)
    pool = torch.zeros(pages, P, Hkv, ROW, dtype=torch.uint8, device="cuda")
    bt = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    zl.kv_append_q4(k, v, pool, bt, sl, page_size=P)
    kk, vv = (x[0].double() for x in zl.kv_read_q4(pool, bt, sl, page_size=P, tokens=L))
    q = (torch.randn(1, 1, Hq, 128, generator=g) * 2).to(torch.bfloat16).cuda()
    lse = torch.empty(1, 1, Hq, device="cuda")
    out = zl.decode_attn_q4(q, pool, bt, sl, page_size=P, scale=SCALE, lse=lse, max_seq_len=L)
    for h in range(Hq):
        x = kk[:, h // 4] @ q[0, 0, h].double() * SCALE
        p = torch.softmax(x, 0)
        o = p @ vv[:, h // 4]
        # roundings as in plain_q4.tolerance; sizes of scores here: below 2^6
        rel = 2.0 ** -11 + 2.0 ** -15
        tol = 2.0 ** -8 * o.abs() + 1.01 * (rel * (p @ vv[:, h // 4].abs())
                                            + L * 2.0 ** -32 * vv.abs().max())
        assert bool(((out[0, 0, h].double() - o).abs() <= tol).all())
        assert abs(float(lse[0, 0, h]) - float(torch.logsumexp(x, 0))) < 2.0 ** -14


def test_4096_sequences():
    B = 4096
    lens = [(7 * i) % 23 for i in range(B)]
    c = Cache(31, lens, 1, 16)
    check(c, queries(c, 1, 2))
