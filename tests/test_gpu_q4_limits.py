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
