"""Attention over a 4-bit cache whose wait runs out: the call reports it, the rows that miss
tokens are zeros, every warp and CTA still meets the barriers it has to, and the next call on
the same buffers is right. The stall is the ZL_DECODE_TEST_STALL hook's (about 50 ms): the
first warp of every CTA gives up on its tiles, with their copies in flight."""
import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_q4 import Cache, attention, bf16
from test_gpu_q4_attn import SCALE, queries

pytestmark = pytest.mark.gpu


class Call:
    """A call by its parameter struct, on buffers of its own."""

    def __init__(self, c, q, **kw):
        pool, bt, sl = c.on_gpu()
        B, q_len, Hq, _ = q.shape
        self.out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, q_len, Hq), 7.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        st = pool.stride()
        p = self.p = zl.DecodeQ4Params()
        p.struct_size = ctypes.sizeof(p)
        qd = q.cuda()
        p.q, p.pool, p.out, p.lse = (x.data_ptr() for x in (qd, pool, self.out, self.lse))
        p.page_stride = st[0]
        p.token_stride, p.head_stride = (st[1], st[2]) if c.layout == "NHD" else (st[2], st[1])
        p.block_table, p.seq_lens, p.err_flags = (x.data_ptr() for x in (bt, sl, self.err))
        p.block_table_stride, p.num_pages, p.page_size = bt.shape[1], c.pages, c.P
        p.B, p.q_len, p.Hq, p.Hkv, p.scale = B, q_len, Hq, c.Hkv, SCALE
        for n, v in kw.items():
            setattr(p, n, v)
        n = ctypes.c_size_t(0)
        assert zl.lib().zl_decode_attn_q4_workspace_size(ctypes.byref(p), ctypes.byref(n)) == zl.OK
        ws = torch.full((max(n.value, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = ws.data_ptr(), n.value
        self.keep = (qd, pool, bt, sl, ws)

    def __call__(self, flags):
        self.p.flags = flags
        self.err.zero_()
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert zl.lib().zl_decode_attn_q4(ctypes.byref(self.p), stream) == zl.OK
        torch.cuda.synchronize()
        return bf16(self.out), bf16(self.lse), int(self.err.item())


CASES = [  # lens, Hq, Hkv, query tokens, arguments
    ([900, 64, 0, 333], 8, 2, 1, dict(num_ctas=7)),             # cut and merged
    ([900, 64, 0, 333], 8, 2, 5, dict(num_ctas=5)),
    ([700, 333, 17, 0, 150], 16, 8, 1, dict(max_seq_len=200000)),  # heads side by side
    ([40, 17, 0, 60], 8, 2, 1, dict(max_seq_len=64)),           # whole units
    ([40, 17, 0, 60], 8, 2, 5, dict(max_seq_len=64)),
    ([700, 0, 33, 1999], 8, 2, 1, dict(max_seq_len=2000)),      # clusters
    ([1500, 40], 5, 1, 3, dict(max_seq_len=1500)),
    ([900], 2, 2, 1, dict(max_seq_len=900)),
]


@pytest.mark.parametrize("lens,Hq,Hkv,q_len,kw", CASES)
def test_a_wait_that_runs_out(lens, Hq, Hkv, q_len, kw):
    c = Cache(90 + q_len, lens, Hkv)
    q = queries(c, q_len, Hq)
    call = Call(c, q, **kw)
    want, want_lse, t_out, t_lse = attention(bf16(q), [c.kv(b) for b in range(len(lens))], lens,
                                             SCALE)

    def right(out, lse):
        none = np.isinf(want_lse)
        near = np.abs(np.where(none, 0, lse) - np.where(none, 0, want_lse)) <= t_lse
        return (np.abs(out - want) <= t_out).all(-1) & np.where(none, lse == -np.inf, near)

    out, lse, err = call(0)
    assert err == 0 and right(out, lse).all()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    cut, cut_lse, err = call(zl.TEST_STALL)
    b.record()
    torch.cuda.synchronize()
    assert err == zl.DEVERR_TIMEOUT and a.elapsed_time(b) < 1000.0
    zero = ~cut.any(-1) & (cut_lse == -np.inf)
    assert (zero | right(cut, cut_lse)).all()
    sees = np.isfinite(want_lse)
    # the first warp has the first kv head's tiles (of each bundle): where a unit is one CTA's
    # or one cluster's, some of every sequence's
    if "num_ctas" in kw or kw["max_seq_len"] == 200000:
        assert (zero & sees).any()
    else:
        assert zero[:, :, :Hq // Hkv].all()
    again, again_lse, err = call(0)
    assert err == 0 and np.array_equal(again, out) and np.array_equal(again_lse, lse)


def test_without_an_error_word():
    c = Cache(99, [300], 2)
    q = queries(c, 1, 4)
    call = Call(c, q, err_flags=None)
    out, lse, _ = call(0)
    call(zl.TEST_STALL)
    again, again_lse, _ = call(0)
    assert np.array_equal(again, out) and np.array_equal(again_lse, lse)
