"""Writing the 4-bit cache and reading it back: every byte against the definition in 64
bits (both roundings are decided exactly, so there is no tolerance)."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_q4 import ROW, Cache, bf16, pack, random_rows, unpack

pytestmark = pytest.mark.gpu


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def put(c, k, v, q_len, new=None, skip=()):
    """The pool after an append, by the definition."""
    for b, L in enumerate(c.lens):
        n = q_len if new is None else new[b]
        if b not in skip and n:
            c.put(b, np.arange(L - n, L), pack(bf16(k[b, :n]), bf16(v[b, :n])))


@pytest.mark.parametrize("lens,Hkv,P,q_len,layout", [
    ([1], 1, 16, 1, "NHD"), ([17, 16, 5], 2, 16, 1, "HND"), ([40, 70, 100], 8, 16, 5, "NHD"),
    ([130, 128, 129, 300], 3, 48, 128, "HND"), ([65, 1000], 5, 64, 65, "NHD"),
    ([33] * 70, 1, 16, 33, "NHD"), ([7, 9], 40, 1, 3, "HND"),
])
def test_append_then_read(lens, Hkv, P, q_len, layout):
    c = Cache(7 * q_len + Hkv, lens, Hkv, P, layout)
    B, n = len(lens), max(lens) + 2
    k, v = random_rows(c.g, B, q_len, Hkv, spread=4.0), random_rows(c.g, B, q_len, Hkv, spread=4.0)
    pool, bt, sl = c.on_gpu()
    err = err_word()
    zl.kv_append_q4(k.cuda(), v.cuda(), pool, bt, sl, page_size=P, layout=layout, err_flags=err)
    put(c, k, v, q_len)
    assert np.array_equal(pool.cpu().numpy(), c.pool)
    ko = torch.full((B, n, Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    zl.kv_read_q4(pool, bt, sl, page_size=P, k_out=ko, v_out=vo, layout=layout, err_flags=err)
    assert int(err.item()) == 0
    for b, L in enumerate(lens):
        for got, want in zip((ko, vo), c.kv(b)):
            assert np.array_equal(bf16(got[b, :L]), want)
            assert bool((got[b, L:] == 7.0).all())  # rows behind the sequence


def test_every_bf16_number_and_every_border():
    """Blocks whose largest is every finite bf16 magnitude, with elements around every
    border of that scale; zeros, subnormals and the largest numbers among them."""
    bits = np.arange(0x7F80, dtype=np.int64)
    top = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)
    six = top.double().numpy() / 6
    x = np.zeros((len(bits), 16))
    x[:, 0] = top.double()
    for j, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        x[:, 1 + 2 * j] = np.minimum(m * six, top.double().numpy())
        x[:, 2 + 2 * j] = -np.minimum(np.nextafter(m * six, 0), top.double().numpy())
    x = torch.from_numpy(x).to(torch.bfloat16)
    # the same with the borders of the rounded scale, which are bf16 numbers
    rows = torch.zeros(-(-len(bits) // 8) * 8, 16, dtype=torch.bfloat16)
    rows[:len(bits)] = x
    rows = rows.view(-1, 1, 1, 128)
    back = unpack(pack(bf16(rows), bf16(rows)))[0].reshape(-1, 16)
    s = np.abs(back).max(-1) / 6  # the scale, where the largest has code 7
    exact = np.zeros((len(back), 16))
    exact[:, 0] = bf16(rows).reshape(-1, 16)[:, 0]
    for j, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        exact[:, 1 + j] = m * s
        exact[:, 8 + j] = -m * s
    exact = np.minimum(np.abs(exact), exact[:, :1]) * np.sign(exact)
    border = torch.from_numpy(exact).to(torch.bfloat16).view(-1, 1, 1, 128)
    for k, v in ((rows, border), (border, -rows)):
        B = len(k)
        pool = torch.zeros(B, 1, 1, ROW, dtype=torch.uint8, device="cuda")
        bt = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
        sl = torch.ones(B, dtype=torch.int32, device="cuda")
        zl.kv_append_q4(k.cuda(), v.cuda(), pool, bt, sl, page_size=1)
        want = pack(bf16(k), bf16(v))
        got = pool.cpu().numpy().reshape(want.shape)
        assert np.array_equal(got, want)
        ko, vo = zl.kv_read_q4(pool, bt, sl, page_size=1, tokens=1)
        wk, wv = unpack(want)
        assert np.array_equal(bf16(ko), wk) and np.array_equal(bf16(vo), wv)


def test_every_byte_reads_back():
    """All codes under all scales, those that writing never makes included."""
    rows = np.zeros((256, ROW), np.uint8)
    rows[:, :128] = np.random.default_rng(3).integers(0, 256, (256, 128))
    rows[:, :8] = np.arange(16, dtype=np.uint8)[None, ::2] | (np.arange(16, dtype=np.uint8)[None, 1::2] << 4)
    rows[:, 128:] = np.arange(256, dtype=np.uint8)[:, None]
    pool = torch.from_numpy(rows.reshape(16, 16, 1, ROW)).cuda()
    bt = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    sl = torch.tensor([256], dtype=torch.int32, device="cuda")
    got = zl.kv_read_q4(pool, bt, sl, page_size=16, tokens=256)
    for x, want in zip(got, unpack(rows)):
        x = bf16(x).reshape(256, 128)
        assert np.array_equal(x[:248], want[:248])
        assert not np.isfinite(x[249:]).any()  # (248: an infinity, NaN where the code is 0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_block_with_a_number_that_is_none(value):
    c = Cache(5, [20, 3], 2)
    k, v = random_rows(c.g, 2, 2, 2), random_rows(c.g, 2, 2, 2)
    k[0, 1, 0, 37] = value
    v[1, 0, 1, 127] = value
    pool, bt, sl = c.on_gpu()
    zl.kv_append_q4(k.cuda(), v.cuda(), pool, bt, sl, page_size=16)
    put(c, k, v, 2)
    assert np.array_equal(pool.cpu().numpy(), c.pool)
    ko, vo = zl.kv_read_q4(pool, bt, sl, page_size=16, tokens=20)
    for b, L in enumerate(c.lens):
        for got, want in zip((ko, vo), c.kv(b)):
            assert np.array_equal(bf16(got[b, :L]), want, equal_nan=True)
    assert np.isnan(bf16(ko[0, 19, 0, 32:48])).all() and np.isfinite(bf16(ko[0, 19, 0, 48:])).all()
    assert np.isnan(bf16(vo[1, 1, 1, 112:])).all()


def test_padded_batch():
    """Every sequence has its own number of new tokens; the padding is not read."""
    lens, new, q_len = [37, 200, 5, 64, 9], [37, 1, 0, 40, 9], 40
    c = Cache(11, lens, 4)
    k, v = random_rows(c.g, 5, q_len, 4), random_rows(c.g, 5, q_len, 4)
    for b, n in enumerate(new):
        k[b, n:] = float("nan")
    pool, bt, sl = c.on_gpu()
    err = err_word()
    zl.kv_append_q4(k.cuda(), v.cuda(), pool, bt, sl, page_size=16, err_flags=err,
                    new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"))
    put(c, k, v, q_len, new)
    assert int(err.item()) == 0 and np.array_equal(pool.cpu().numpy(), c.pool)


def test_bad_lengths_and_pages():
    lens = [37, 200, 5, 64, 9, 30]
    c = Cache(12, lens, 2)
    k, v = random_rows(c.g, 6, 8, 2), random_rows(c.g, 6, 8, 2)
    pool, bt, sl = c.on_gpu()
    args = dict(page_size=16)
    before = pool.clone()

    def append(sl, new, want):
        err = err_word()
        zl.kv_append_q4(k.cuda(), v.cuda(), pool, bt, torch.tensor(sl, dtype=torch.int32).cuda(),
                        new_lens=torch.tensor(new, dtype=torch.int32).cuda(), err_flags=err, **args)
        assert int(err.item()) == want

    append([7, -1, 10000, 1 << 30, 0, 3], [8, 8, 8, 8, 1, 4], zl.DEVERR_BAD_SEQ_LEN)
    append(lens, [9, -1, 6, 1 << 30, -8, 31], zl.DEVERR_BAD_SEQ_LEN)
    assert torch.equal(pool, before)
    # a new token on a page that is none: that token alone is left out
    bt[0, 2], bt[3, 3] = c.pages, -1
    append(lens, [8, 8, 0, 3, 8, 8], zl.DEVERR_BAD_PAGE)
    good = [8, 8, 0, 0, 8, 8]
    # (tokens 32 .. 36 of sequence 0 lie on the bad page, 29 .. 31 do not)
    put(c, k, v, 8, good, skip=(0,))
    c.put(0, np.arange(29, 32), pack(bf16(k[0, :3]), bf16(v[0, :3])))
    assert np.array_equal(pool.cpu().numpy(), c.pool)
    # reading: rows on a bad page, and sequences with bad lengths, are left as they were
    ko = torch.full((6, 200, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    vo, err = ko.clone(), err_word()
    sl = torch.tensor([37, 201, -3, 64, 9, 30], dtype=torch.int32, device="cuda")
    zl.kv_read_q4(pool, bt, sl, k_out=ko, v_out=vo, err_flags=err, **args)
    assert int(err.item()) == zl.DEVERR_BAD_SEQ_LEN | zl.DEVERR_BAD_PAGE
    assert bool((ko[1:3] == 3).all()) and bool((vo[0, 32:] == 3).all())
    assert bool((vo[3, 48:] == 3).all())
    for b, L in ((0, 32), (3, 48), (4, 9), (5, 30)):
        want = unpack(c.rows(b, np.arange(L)))
        assert np.array_equal(bf16(ko[b, :L]), want[0]) and np.array_equal(bf16(vo[b, :L]), want[1])


def test_slices_of_a_projection_and_16_byte_rows():
    """Strided new rows, and ones that start 16 bytes off a 32-byte boundary."""
    B, n, Hkv = 3, 4, 2
    for off, width in ((0, 10 * 128), (8, 10 * 128 + 8), (8, 10 * 128 + 16)):
        c = Cache(13 + off + width, [30, 4, 17], Hkv)
        buf = torch.zeros(B, n, width, dtype=torch.bfloat16)
        kv = random_rows(c.g, B, n, 2 * Hkv)
        buf[..., off:off + 4 * 128] = kv.flatten(2)
        d = buf.cuda()
        k = d[..., off:off + 256].unflatten(-1, (2, 128))
        v = d[..., off + 256:off + 512].unflatten(-1, (2, 128))
        pool, bt, sl = c.on_gpu()
        zl.kv_append_q4(k, v, pool, bt, sl, page_size=16)
        put(c, kv[:, :, :2], kv[:, :, 2:], n)
        assert np.array_equal(pool.cpu().numpy(), c.pool)


def test_pages_beyond_2_31_bytes():
    """A pool whose pages lie far apart: offsets pass 32 bits."""
    P, Hkv = 16, 2
    far = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
    step = (5 << 30) // 4 // 16 * 16
    pool = far.as_strided((4, P, Hkv, ROW), (step, Hkv * ROW, ROW, 1))
    c = Cache(17, [60], Hkv, spare=0, fill=False)
    pool.copy_(torch.from_numpy(c.pool))
    k, v = random_rows(c.g, 1, 60, Hkv), random_rows(c.g, 1, 60, Hkv)
    _, bt, sl = c.on_gpu()
    zl.kv_append_q4(k.cuda(), v.cuda(), pool, bt, sl, page_size=P)
    put(c, k, v, 60)
    assert np.array_equal(pool.cpu().numpy(), c.pool)
    ko, vo = zl.kv_read_q4(pool, bt, sl, page_size=P, tokens=60)
    assert np.array_equal(bf16(ko[0]), c.kv(0)[0]) and np.array_equal(bf16(vo[0]), c.kv(0)[1])


def test_one_of_the_two_outputs():
    c = Cache(18, [20, 0], 2)
    pool, bt, sl = c.on_gpu()
    ko = torch.zeros(2, 20, 2, 128, dtype=torch.bfloat16, device="cuda")
    assert zl.kv_read_q4(pool, bt, sl, page_size=16, k_out=ko)[1] is None
    assert np.array_equal(bf16(ko[0]), c.kv(0)[0]) and not bool(ko[1].any())
    vo = torch.zeros_like(ko)
    zl.kv_read_q4(pool, bt, sl, page_size=16, v_out=vo)
    assert np.array_equal(bf16(vo[0]), c.kv(0)[1])


def test_eviction_and_commit_move_its_rows():
    """The pool as a latent-only bf16 pool of 72 elements per row."""
    c = Cache(19, [50, 20], 3)
    pool, bt, sl = c.on_gpu()
    rows = pool.view(torch.bfloat16)
    path = torch.tensor([[0, 2, 3], [1, 0, 0]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    sl = zl.kv_commit(rows, None, bt, sl, path, acc, page_size=16, q_len=6)
    assert sl.tolist() == [47, 15]
    for b, taken in ((0, [0, 2, 3]), (1, [1])):
        first = c.lens[b] - 6
        c.put(b, np.arange(first, first + len(taken)), c.rows(b, first + np.array(taken)).copy())
    assert np.array_equal(pool.cpu().numpy(), c.pool)
    w = torch.rand(2, 3, 47, device="cuda")
    new, kept = zl.kv_evict(rows, None, bt, sl, w, page_size=16, budget=20)
    assert new.tolist() == [20, 15]
    old = c.rows(0, np.arange(47)).copy()
    for h in range(3):
        want = old[kept[0, h].cpu().numpy(), h]
        page, slot = c.place(0, np.arange(20))
        c.pool[page, slot, h] = want
    assert np.array_equal(pool.cpu().numpy(), c.pool)
