"""How large a call over a 4-bit cache may be: what the header promises is accepted, and the
line of tiles that one CTA could not count is refused. (Workspace queries: nothing is launched.
They ask the device for its SMs.)"""
import ctypes

import pytest

import paged_decode_attention_gqa_gb300 as zl
from test_q4_abi import _decode

pytestmark = pytest.mark.gpu


def query(**kw):
    n = ctypes.c_size_t(0)
    return zl.lib().zl_decode_attn_q4_workspace_size(ctypes.byref(_decode(**kw)), ctypes.byref(n))


def promised(B, q_len, Hq, Hkv, reach, num_ctas):
    """The header's bounds, the plain ones taken as kept."""
    groups = -(-(Hq // Hkv * q_len) // 16)
    n = (reach // 32 + 33) * Hkv * groups
    return n < 1 << 29 and B * n < (num_ctas or 152) << 29


BIG = dict(B=4096, q_len=128, Hq=64, Hkv=8, page_size=16, block_table_stride=8192)


def test_a_line_that_one_cta_cannot_count_is_refused():
    """Inside the bounds on tiles and heads: 2^25 tiles of 16, 2^28 with the heads."""
    assert not promised(4096, 128, 64, 8, 8192 * 16, 1)
    assert query(num_ctas=1, **BIG) == zl.ERR_UNSUPPORTED
    assert query(num_ctas=0, **BIG) == query(num_ctas=1000, **BIG) == zl.OK
    # one sequence's own line
    far = dict(B=1, q_len=128, Hq=128 * 127, Hkv=127, page_size=1024)
    assert not promised(1, 128, 128 * 127, 127, 1024 << 14, 0)
    assert query(block_table_stride=1 << 14, **far) == zl.ERR_UNSUPPORTED


@pytest.mark.parametrize("num_ctas", [0, 1, 3, 152, 65535])
@pytest.mark.parametrize("max_seq_len", [0, 1, 100, 5000, 1 << 20])
def test_what_the_header_promises_is_accepted(num_ctas, max_seq_len):
    seen = 0
    for B in (1, 7, 512, 4096):
        for q_len, g in ((1, 1), (1, 9), (5, 4), (128, 128)):
            for Hkv in (1, 7, 8, 61, 128):
                for stride in (1, 100, 8192, 1 << 17, 1 << 21, 1 << 24, 1 << 27):
                    tiles = B * stride
                    if tiles >= 1 << 31 or tiles * Hkv >= 1 << 40:
                        continue
                    if not promised(B, q_len, g * Hkv, Hkv, stride * 16, num_ctas):
                        continue
                    seen += 1
                    assert query(B=B, q_len=q_len, Hq=g * Hkv, Hkv=Hkv, page_size=16,
                                 block_table_stride=stride, num_ctas=num_ctas,
                                 max_seq_len=max_seq_len) == zl.OK, (B, q_len, g, Hkv, stride)
    assert seen > 100


@pytest.mark.parametrize("L", [(1 << 31) - 32, (1 << 31) - 31, (1 << 31) - 1])
def test_the_longest_sequences(L):
    """Up to the last length that 32 bits hold, over four pages mapped again and again: K is
    0, so the output is the mean of V over the tokens. A warp adds some 2^15 tiles in 32 bits,
    two steps each, which may be off by 2^-23 of the sum so far: 2^-7 of the mean magnitude."""
    import numpy as np
    import torch
    from plain_q4 import bf16, pack, random_rows, unpack

    P, g = 1024, np.random.default_rng(9)
    rows = np.stack([pack(np.zeros((P, 1, 128)), bf16(random_rows(g, P, 1))) for _ in range(4)])
    v = unpack(rows)[1][:, :, 0]                      # [4, P, 128]
    pool = torch.from_numpy(rows).cuda()
    pages = torch.arange(1 << 21, dtype=torch.int32, device="cuda")[None] % 4
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    lse = torch.zeros(1, 2, 3, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, 3, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = zl.decode_attn_q4(q, pool, pages.contiguous(), sl, page_size=P, scale=0.1, lse=lse,
                            err_flags=err)
    assert int(err.item()) == 0
    whole, rest = divmod(L, 4 * P)
    every, some = v.reshape(4 * P, 128), v.reshape(4 * P, 128)[:rest]
    want = (whole * every.sum(0) + some.sum(0)) / L
    size = (whole * np.abs(every).sum(0) + np.abs(some).sum(0)) / L
    assert (np.abs(bf16(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * size).all()
    assert np.abs(bf16(lse) - np.log(L)).max() <= 2.0 ** -16
