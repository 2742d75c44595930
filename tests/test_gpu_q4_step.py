"""The operators around the 4-bit cache as a decode loop uses them: prompts, steps,
drafted tokens, graphs, streams, overlapping calls."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_q4 import ROW, attention, bf16, norm_rope, pack, unpack

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


class Model:
    """One attention layer's state: weights of the norms, a rotation, a pool, tables."""

    def __init__(self, seed, B, Hq, Hkv, P, longest, layout="NHD"):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.P, self.layout = B, Hq, Hkv, P, layout
        width = -(-longest // P)
        pages = B * width + 2
        shape = (pages, P, Hkv, ROW) if layout == "NHD" else (pages, Hkv, P, ROW)
        self.pool = torch.randint(0, 256, shape, dtype=torch.uint8, generator=self.g).cuda()
        self.bt = torch.randperm(pages, generator=self.g)[:B * width].view(B, width)
        self.bt = self.bt.to(torch.int32).cuda()
        self.w = (torch.rand(2, 128, generator=self.g) + 0.5).cuda()
        self.freq = zl.rope_frequencies(128, 1e6)
        self.rope = zl.Rope(self.freq)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def projection(self, n):
        x = torch.randn(self.B, n, self.Hq + 2 * self.Hkv, 128, generator=self.g) * 2
        return x.to(torch.bfloat16).cuda()

    def norm(self, qkv, lens, **kw):
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], 2)
        return zl.qk_norm_rope(q, k, v=v, rope=self.rope, q_weight=self.w[0], k_weight=self.w[1],
                               pool=self.pool, block_table=self.bt, seq_lens=lens,
                               page_size=self.P, layout=self.layout, err_flags=self.err, **kw)[0]

    def attend(self, q, lens, **kw):
        return zl.decode_attn_q4(q, self.pool, self.bt, lens, page_size=self.P, scale=SCALE,
                                 layout=self.layout, err_flags=self.err, **kw)

    def plain_rows(self, qkv, lens):
        """What the cache must hold of these tokens, and the queries, by the formulas in 64
        bits rounded to bf16 where the kernel rounds; with them which rows that decides: a
        key within 2^-16 of a border between two bf16 numbers may round either way."""
        n = qkv.shape[1]
        q, k, v = (bf16(x) for x in qkv.split([self.Hq, self.Hkv, self.Hkv], 2))
        pos = np.array(lens)[None, :, None] - n + np.arange(n)
        w = bf16(self.w)
        rot = [0] * 64
        q = norm_rope(q, w[0], 1e-6, pos, self.freq, rot, False)
        k = norm_rope(k, w[1], 1e-6, pos, self.freq, rot, False)
        return q, k, v


def lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_prompt_then_steps(layout):
    """A ragged prompt, then steps of 1 and 3 tokens: cache and outputs against the plain
    forms fed with the cache's own values."""
    B, Hq, Hkv, P = 3, 8, 2, 16
    m = Model(1, B, Hq, Hkv, P, 200, layout)
    new = [40, 7, 100]
    n = max(new)
    qkv = m.projection(n)
    # a ragged prompt: norms and rotation of the padded batch at positions 0 .., then the
    # valid rows are stored
    q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, n).contiguous()
    _, kn = zl.qk_norm_rope(q, k, rope=m.rope, positions=pos, q_weight=m.w[0], k_weight=m.w[1])
    lens = lengths(new)
    zl.kv_append_q4(kn, v, m.pool, m.bt, lens, page_size=P, new_lens=lens, layout=layout,
                    err_flags=m.err)
    want = [(bf16(kn[b, :L]), bf16(v[b, :L])) for b, L in enumerate(new)]
    for count in (1, 3, 1):
        qkv = m.projection(count)
        lens = lens + count
        L = lens.tolist()
        qn = m.norm(qkv, lens)
        out = m.attend(qn, lens, lse=(lse := torch.empty(B, count, Hq, device="cuda")))
        # the same step in two launches
        _, k, v = qkv.split([Hq, Hkv, Hkv], 2)
        at = (lens[:, None] - count + torch.arange(count, device="cuda")).to(torch.int32)
        q2, k2 = zl.qk_norm_rope(qkv[:, :, :Hq], k, rope=m.rope, positions=at, q_weight=m.w[0],
                                 k_weight=m.w[1])
        assert torch.equal(q2, qn)
        want = [(np.concatenate([a, bf16(k2[b])]), np.concatenate([c, bf16(v[b])]))
                for b, (a, c) in enumerate(want)]
        ko, vo = zl.kv_read_q4(m.pool, m.bt, lens, page_size=P, tokens=max(L), layout=layout)
        held = [unpack(pack(a, c)) for a, c in want]
        for b in range(B):
            assert np.array_equal(bf16(ko[b, :L[b]]), held[b][0])
            assert np.array_equal(bf16(vo[b, :L[b]]), held[b][1])
        o, l, t_o, t_l = attention(bf16(qn), held, L, SCALE)
        assert (np.abs(bf16(out) - o) <= t_o).all() and (np.abs(bf16(lse) - l) <= t_l).all()
    assert int(m.err.item()) == 0


def test_norms_feed_the_cache_within_a_bf16_step():
    """The stored keys against the formula: the key's own rounding, then the block's: a
    value lies within half a step of the coarser of the two codes around it."""
    m = Model(2, 4, 4, 2, 32, 64)
    qkv = m.projection(5)
    L = [5, 20, 33, 64]
    qn = m.norm(qkv, lengths(L))
    q, k, v = m.plain_rows(qkv, L)
    assert (np.abs(bf16(qn) - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -17 * np.abs(q).max()).all()
    ko, _ = zl.kv_read_q4(m.pool, m.bt, lengths(L), page_size=32, tokens=64)
    for b in range(4):
        got = bf16(ko[b, L[b] - 5:L[b]]).reshape(5, 2, 8, 16)
        ref = k[b].reshape(5, 2, 8, 16)
        top = np.abs(ref).max(-1, keepdims=True)
        # a scale is at most top / 6 * (1 + 2^-4) and a step of codes 2 scales: half of it,
        # and beyond 6 scales at most 2^-4 of the largest
        assert (np.abs(got - ref) <= top / 6 * (1 + 2.0 ** -4) + 2.0 ** -7 * top).all()


@pytest.mark.parametrize("filled", [False, True])
def test_a_step_captured_in_a_graph(filled):
    """Norm and store, attention (cut and merged), replayed over growing sequences with new
    inputs in the same buffers; a second graph of another shape in between. The cache holds
    any bytes (NaN scales among them: compared as bits), or cached tokens."""
    B, Hq, Hkv, P = 4, 16, 4, 16
    m = Model(3, B, Hq, Hkv, P, 700)
    lens = lengths([600, 30, 333, 1])
    if filled:
        k = torch.randn(B, 600, Hkv, 128, generator=m.g).to(torch.bfloat16).cuda()
        zl.kv_append_q4(k, k, m.pool, m.bt, lens, page_size=P, new_lens=lens)
    qkv = m.projection(1)
    start = m.pool.clone()
    out = torch.empty(B, 1, Hq, 128, dtype=torch.bfloat16, device="cuda")
    small = lengths([3, 3, 3, 3])
    other = torch.empty_like(out)

    def step():
        m.attend(m.norm(qkv, lens), lens, out=out)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        m.attend(qkv[:, :, :Hq].contiguous(), small, out=other)
    stream.synchronize()
    graphs = []
    for fn in (step, lambda: m.attend(qkv[:, :, :Hq].contiguous(), small, out=other)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            fn()
        graphs.append(g)
    m.pool.copy_(start)
    inputs = [m.projection(1) for _ in range(4)]
    got = []
    for x in inputs:
        qkv.copy_(x)
        graphs[0].replay()
        got.append(out.clone())
        graphs[1].replay()
        lens += 1
    torch.cuda.synchronize()
    m.pool.copy_(start)
    lens -= len(inputs)
    for x, y in zip(inputs, got):
        qkv.copy_(x)
        x = m.attend(m.norm(qkv, lens), lens)
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert not filled or bool(torch.isfinite(x).all())
        lens += 1
    assert int(m.err.item()) == 0


def test_calls_on_two_streams_at_once():
    """Overlapping calls take scratch of their own."""
    B, Hq, Hkv, P = 2, 8, 2, 16
    models = [Model(10 + i, B, Hq, Hkv, P, 3000) for i in range(2)]
    lens = lengths([2999, 1500])
    qs = [torch.randn(B, 1, Hq, 128, generator=m.g).to(torch.bfloat16).cuda() for m in models]
    for m in models:  # finite contents
        k = torch.randn(B, 2999, Hkv, 128, generator=m.g).to(torch.bfloat16).cuda()
        zl.kv_append_q4(k, k, m.pool, m.bt, lens, page_size=P, new_lens=lens)
    want = [m.attend(q, lens) for m, q in zip(models, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in models]
    got = [[], []]
    for _ in range(20):
        for i, (m, q, s) in enumerate(zip(models, qs, streams)):
            got[i].append(m.attend(q, lens, stream=s))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(w, x) for x in many)


def test_a_workspace_of_the_exact_size_and_one_too_small():
    m = Model(20, 2, 8, 2, 16, 2000)
    lens = lengths([1999, 800])
    k = torch.randn(2, 1999, 2, 128, generator=m.g).to(torch.bfloat16).cuda()
    zl.kv_append_q4(k, k, m.pool, m.bt, lens, page_size=16, new_lens=lens)
    q = torch.randn(2, 1, 8, 128, generator=m.g).to(torch.bfloat16).cuda()
    want = m.attend(q, lens)
    import ctypes
    p = zl.DecodeQ4Params()
    p.struct_size = ctypes.sizeof(p)
    p.B, p.q_len, p.Hq, p.Hkv, p.page_size, p.num_pages = 2, 1, 8, 2, 16, m.pool.shape[0]
    p.block_table_stride, p.scale = m.bt.stride(0), SCALE
    n = ctypes.c_size_t(0)
    assert zl.lib().zl_decode_attn_q4_workspace_size(ctypes.byref(p), ctypes.byref(n)) == zl.OK
    buf = torch.full((n.value + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = buf[:n.value]
    assert torch.equal(m.attend(q, lens, workspace=ws), want)
    assert bool((buf[n.value:] == 0xFF).all())
    with pytest.raises(zl.ZlError) as e:
        m.attend(q, lens, workspace=buf[:n.value - 256])
    assert e.value.status == zl.ERR_WORKSPACE


def test_a_bound_that_does_not_hold_changes_nothing():
    """max_seq_len sizes the grid only: too small a one gives the same result within
    rounding (the units are then not cut)."""
    m = Model(21, 3, 8, 2, 16, 1200)
    lens = lengths([1200, 3, 700])
    k = torch.randn(3, 1200, 2, 128, generator=m.g).to(torch.bfloat16).cuda()
    zl.kv_append_q4(k, k, m.pool, m.bt, lens, page_size=16, new_lens=lens)
    for n in (1, 4):
        q = torch.randn(3, n, 8, 128, generator=m.g).to(torch.bfloat16).cuda()
        a, b = m.attend(q, lens), m.attend(q, lens, max_seq_len=4)
        # each is within bf16's half step of the same sum, and fp16's of P
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -8)


def test_rows_and_cache_of_other_sequences_stay():
    """A step of some sequences leaves every byte of the pool that is not theirs."""
    m = Model(22, 3, 4, 2, 16, 64)
    before = m.pool.clone()
    qkv = m.projection(2)
    lens = lengths([33, 17, 64])
    m.norm(qkv, lens)
    changed = (m.pool != before).any(-1).nonzero().tolist()
    mine = set()
    for b, L in enumerate(lens.tolist()):
        for t in (L - 2, L - 1):
            for h in range(2):
                mine.add((int(m.bt[b, t // 16]), t % 16, h))
    assert {tuple(x) for x in changed} <= mine and len(changed) >= len(mine) - 1


@pytest.mark.parametrize("graph", [False, True])
def test_calls_that_follow_one_another_without_a_wait(graph):
    """Each call reads what the one before it wrote: norm, attention, append of its output,
    read-back, norm of that. The bits are those of calls that are waited for."""
    B, Hq, Hkv, P, n = 3, 8, 4, 16, 2
    m = Model(40, B, Hq, Hkv, P, 900)
    lens = lengths([900, 77, 410])
    k = torch.randn(B, 900, Hkv, 128, generator=m.g).to(torch.bfloat16).cuda()
    zl.kv_append_q4(k, k, m.pool, m.bt, lens, page_size=P, new_lens=lens)
    first, start = m.projection(n), m.pool.clone()
    qkv, q = torch.empty_like(first), torch.empty(B, n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    back = torch.zeros(2, B, 900, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    positions = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)

    def steps(after):
        for _ in range(6):
            m.norm(qkv, lens, q_out=q)
            after()
            m.attend(q, lens, out=out)
            after()
            zl.kv_append_q4(out[:, :, :Hkv], out[:, :, Hkv:], m.pool, m.bt, lens, page_size=P)
            after()
            zl.kv_read_q4(m.pool, m.bt, lens, k_out=back[0], v_out=back[1], page_size=P)
            after()
            # rows that were read (the newest of one sequence among them) go into the next step
            zl.qk_norm_rope(back[0, :, 75:75 + n].contiguous(), back[1, :, 75:75 + n].contiguous(),
                            rope=m.rope, positions=positions, q_out=qkv[:, :, Hq:Hq + Hkv],
                            k_out=qkv[:, :, Hq + Hkv:])
            after()

    def run(after, g=None):
        qkv.copy_(first)
        m.pool.copy_(start)
        back.zero_()
        torch.cuda.synchronize()
        g.replay() if g else steps(after)
        torch.cuda.synchronize()
        return [x.clone() for x in (qkv, q, out, back, m.pool)]

    want = run(torch.cuda.synchronize)
    g = None
    if graph:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            steps(lambda: None)
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            steps(lambda: None)
    for _ in range(5):
        for a, b in zip(want, run(lambda: None, g)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(m.err.item()) == 0 and bool(torch.isfinite(want[2]).all())
