"""Norm and rotation of queries and keys against the formula in 64 bits (tolerance:
plain_q4.norm_rope_tolerance), and what they store in a cache, byte for byte."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_q4 import Cache, bf16, norm_rope, norm_rope_tolerance

pytestmark = pytest.mark.gpu
EPS = 1e-6


def projection(seed, B, n, Hq, Hkv, size=3.0):
    """q, k, v as slices of one projection's output."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, n, Hq + 2 * Hkv, 128, generator=g) * size
    x = x.to(torch.bfloat16).cuda()
    return x.split([Hq, Hkv, Hkv], 2)


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(2, 128, generator=g) + 0.5).cuda().unbind()


def want(x, w, pos, freq, axis_of=None, interleaved=False, scale=1.0, eps=EPS):
    """The formula's rows and how far the kernel's may be off."""
    x = bf16(x)
    w = None if w is None else bf16(w)
    axis_of = [0] * len(freq) if axis_of is None else axis_of
    y = norm_rope(x, w, eps, pos, freq, axis_of, interleaved, scale)
    # a pair's size: both elements before the rotation
    size = norm_rope(x, w, eps, pos, [], [], interleaved)
    size = np.abs(size)
    n = len(freq)
    if n:
        one, two = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved
                    else (slice(0, n), slice(n, 2 * n)))
        both = (size[..., one] + size[..., two]) * max(1.0, abs(scale))
        size[..., one] = size[..., two] = both
    return y, norm_rope_tolerance(y, size)


def close(got, ref):
    y, tol = ref
    worst = (np.abs(bf16(got) - y) - tol).max()
    assert worst <= 0, worst


@pytest.mark.parametrize("B,n,Hq,Hkv,rot,interleaved", [
    (1, 1, 1, 1, 128, False), (3, 1, 8, 2, 128, True), (2, 5, 32, 8, 64, False),
    (1, 300, 5, 1, 32, False), (4, 7, 12, 6, 96, True), (2, 33, 16, 4, 96, False),
    (70, 9, 3, 3, 128, False), (1, 2500, 4, 4, 128, True), (2, 3, 100, 50, 32, True),
    (1, 6000, 2, 1, 128, False),
])
def test_shapes(B, n, Hq, Hkv, rot, interleaved):
    q, k, _ = projection(B * 100 + n, B, n, Hq, Hkv)
    qw, kw = weights(n)
    freq = zl.rope_frequencies(rot, 1e6)
    pos = torch.randint(-5, 200000, (B, n), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(n))
    rope = zl.Rope(freq, interleaved=interleaved)
    qo, ko = zl.qk_norm_rope(q, k, rope=rope, positions=pos.cuda(), q_weight=qw, k_weight=kw,
                             eps=EPS)
    assert qo.is_contiguous() and ko.is_contiguous()
    p = pos.numpy()[None]
    close(qo, want(q, qw, p, freq, None, interleaved))
    close(ko, want(k, kw, p, freq, None, interleaved))


def test_without_norm_without_rotation_with_neither():
    q, k, _ = projection(1, 2, 9, 4, 2)
    qw, kw = weights(1)
    pos = torch.arange(18, dtype=torch.int32).view(2, 9)
    freq = zl.rope_frequencies(64, 500.0)
    a = zl.qk_norm_rope(q, k, rope=zl.Rope(freq, scale=1.25), positions=pos.cuda())
    close(a[0], want(q, None, pos.numpy()[None], freq, scale=1.25))
    close(a[1], want(k, None, pos.numpy()[None], freq, scale=1.25))
    a = zl.qk_norm_rope(q, k, q_weight=qw, eps=0.5)
    close(a[0], want(q, qw, None, [], eps=0.5))
    assert torch.equal(a[1], k)
    a = zl.qk_norm_rope(q, k)
    assert torch.equal(a[0], q) and torch.equal(a[1], k)


@pytest.mark.parametrize("axes", [[0] * 16 + [1] * 24 + [2] * 24, [i % 3 for i in range(64)],
                                  [3] * 64])
def test_several_axes(axes):
    B, n = 2, 40
    q, k, _ = projection(2, B, n, 6, 2)
    qw, kw = weights(2)
    freq = zl.rope_frequencies(128, 1e6)
    g = np.random.default_rng(2)
    pos = g.integers(0, 5000, (max(axes) + 1, B, n)).astype(np.int32)
    qo, ko = zl.qk_norm_rope(q, k, rope=zl.Rope(freq, axes=axes), q_weight=qw, k_weight=kw,
                             positions=torch.from_numpy(pos).cuda())
    close(qo, want(q, qw, pos, freq, axes))
    close(ko, want(k, kw, pos, freq, axes))


def test_far_positions_and_odd_frequencies():
    """The angle is exact for every position: also where a 32-bit angle would hold no
    digit of the turn. (The reference multiplies with 64 bits of mantissa.)"""
    if np.finfo(np.longdouble).nmant < 63:
        # 2^31 times a frequency: 53 bits leave an angle of 2^-22 at 2^31 radians
        far = [0, 1, -1, 1 << 20, (1 << 24) + 1, 123456789 >> 4]
    else:
        far = [0, 1, -1, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), 123456789]
    pos = torch.tensor([far], dtype=torch.int32)
    q, k, _ = projection(3, 1, len(far), 2, 1)
    freq = [1.0, -1.0, 3.14159, 1e-9, 0.0, 2.5e-5, 7.0, 1e-3] * 4
    qo, _ = zl.qk_norm_rope(q, k, rope=zl.Rope(freq), positions=pos.cuda())
    close(qo, want(q, None, pos.numpy()[None], freq))


def test_zero_rows_and_numbers_that_are_none():
    q, k, _ = projection(4, 1, 3, 4, 2)
    q, k = q.clone(), k.clone()
    q[0, 0], k[0, 1] = 0, 0
    k[0, 0, 1] = torch.finfo(torch.bfloat16).tiny
    q[0, 2, 3, 7], k[0, 2, 0, 100] = float("nan"), float("inf")
    qw, kw = weights(4)
    rope = zl.Rope(zl.rope_frequencies())
    pos = torch.tensor([[3, 4, 5]], dtype=torch.int32, device="cuda")
    qo, ko = zl.qk_norm_rope(q, k, rope=rope, positions=pos, q_weight=qw, k_weight=kw, eps=EPS)
    assert not qo[0, 0].any() and not ko[0, 1].any()
    assert bool(torch.isnan(qo[0, 2, 3]).all()) and bool(torch.isnan(ko[0, 2, 0]).any())
    assert bool(torch.isfinite(qo[0, :, :3]).all()) and bool(torch.isfinite(ko[0, :, 1]).all())
    close(ko[:, :1], want(k[:, :1], kw, np.array([[[3]]]), zl.rope_frequencies()))


def test_in_place():
    q, k, v = projection(5, 3, 5, 8, 2)
    qw, kw = weights(5)
    rope = zl.Rope(zl.rope_frequencies(64))
    pos = torch.arange(15, dtype=torch.int32, device="cuda").view(3, 5)
    args = dict(rope=rope, positions=pos, q_weight=qw, k_weight=kw)
    a, b = zl.qk_norm_rope(q, k, **args)
    was = v.clone()
    zl.qk_norm_rope(q, k, q_out=q, k_out=k, **args)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, was)


@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("lens,n,Hq,Hkv,P,layout,rot,interleaved", [
    ([1, 40, 17], 1, 8, 2, 16, "NHD", 128, False), ([40, 70, 100], 4, 8, 8, 16, "HND", 64, False),
    ([33, 200], 33, 5, 1, 48, "NHD", 96, False), ([33, 200], 9, 6, 3, 16, "HND", 128, True),
    ([64] * 30, 1, 4, 4, 16, "NHD", 32, False), ([500, 501], 300, 4, 2, 16, "NHD", 96, True),
])
def test_store_equals_the_two_steps(kind, lens, n, Hq, Hkv, P, layout, rot, interleaved):
    """Into a cache in one launch: the bytes of norm and rotation followed by an append."""
    c = Cache(n + Hq, lens, Hkv, P, layout)
    B = len(lens)
    q, k, v = projection(6, B, n, Hq, Hkv)
    k = k.clone()  # (its own strides)
    k[-1, 0, 0, :16] = 0
    qw, kw = weights(6)
    rope = zl.Rope(zl.rope_frequencies(rot), interleaved=interleaved)
    pool, bt, sl = c.on_gpu()
    pos = (sl[:, None] - n + torch.arange(n, dtype=torch.int32, device="cuda")).to(torch.int32)
    args = dict(rope=rope, q_weight=qw, k_weight=kw)
    a, b = zl.qk_norm_rope(q, k, positions=pos, **args)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    where = dict(block_table=bt, seq_lens=sl, page_size=P, layout=layout, err_flags=err)
    if kind == "q4":
        two = pool.clone()
        zl.kv_append_q4(b, v, two, bt, sl, page_size=P, layout=layout)
        qo, ko = zl.qk_norm_rope(q, k, v=v, pool=pool, **where, **args)
        assert torch.equal(pool, two)
    else:
        shape = (*pool.shape[:3], 128)
        kp = torch.randn(shape, device="cuda").to(torch.bfloat16)
        vp = torch.randn(shape, device="cuda").to(torch.bfloat16)
        k2, v2 = kp.clone(), vp.clone()
        zl.kv_append(b, v.contiguous(), k2, v2, bt, sl, page_size=P, layout=layout)
        qo, ko = zl.qk_norm_rope(q, k, v=v, k_pool=kp, v_pool=vp, **where, **args)
        assert torch.equal(kp, k2) and torch.equal(vp, v2)
    assert torch.equal(qo, a) and ko is None and int(err.item()) == 0
    # with k_out as well
    ko = torch.empty(B, n, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    zl.qk_norm_rope(q, k, v=v, pool=pool, k_out=ko, **where, **args)
    assert torch.equal(ko, b)


def test_values_are_stored_bit_for_bit():
    """NaN payloads and negative zeros among the values, into bf16 pools."""
    c = Cache(7, [20, 30], 2)
    q, k, v = projection(7, 2, 3, 2, 2)
    v = torch.randint(-32768, 32768, (2, 3, 2, 128), dtype=torch.int16, device="cuda")
    _, bt, sl = c.on_gpu()
    kp = torch.zeros(c.pages, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    zl.qk_norm_rope(q, k, v=v.view(torch.bfloat16), k_pool=kp, v_pool=vp, block_table=bt,
                    seq_lens=sl, page_size=16)
    for b, L in enumerate(c.lens):
        got = c.rows(b, np.arange(L - 3, L), vp.view(torch.int16).cpu().numpy())
        assert np.array_equal(got, v[b].cpu().numpy())


def test_bad_lengths_and_pages():
    c = Cache(8, [20, 30, 10, 40], 2)
    q, k, v = projection(8, 4, 3, 4, 2)
    pool, bt, sl = c.on_gpu()
    bt[1, 1] = c.pages
    sl[0], sl[3] = 2, 1000
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    two = pool.clone()
    qo, _ = zl.qk_norm_rope(q, k, v=v, pool=pool, block_table=bt, seq_lens=sl, page_size=16,
                            positions=pos, err_flags=err, k_out=(ko := torch.empty_like(
                                k.contiguous())))
    assert int(err.item()) == zl.DEVERR_BAD_SEQ_LEN | zl.DEVERR_BAD_PAGE
    assert torch.equal(qo, q) and torch.equal(ko, k)
    err.zero_()
    zl.kv_append_q4(k, v, two, bt, sl, page_size=16, err_flags=err)
    assert torch.equal(pool, two) and int(err.item()) == 3
    assert np.array_equal(c.rows(0, np.arange(20), pool.cpu().numpy()), c.rows(0, np.arange(20)))


def test_many_tokens_of_a_long_prompt_into_a_cache():
    """One sequence's 5000 tokens at once, the prompt of a step to come."""
    n = 5000
    c = Cache(9, [n], 2, 64, fill=False)
    q, k, v = projection(9, 1, n, 4, 2)
    qw, kw = weights(9)
    pool, bt, sl = c.on_gpu()
    rope = zl.Rope(zl.rope_frequencies(128, 1e6))
    zl.qk_norm_rope(q, k, rope=rope, q_weight=qw, k_weight=kw, v=v, pool=pool, block_table=bt,
                    seq_lens=sl, page_size=64)
    two = torch.from_numpy(c.pool).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    _, b = zl.qk_norm_rope(q, k, rope=rope, q_weight=qw, k_weight=kw, positions=pos)
    zl.kv_append_q4(b, v, two, bt, sl, page_size=64)
    assert torch.equal(pool, two)
