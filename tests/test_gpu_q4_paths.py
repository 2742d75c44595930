"""Which way a call over a 4-bit cache goes (cut and merged, a CTA to a unit, a cluster to a
unit), read from the kernels that a captured graph of it holds, with the results of each; and
clusters in graphs and on two streams.

Expected ways are those of a device of 152 SMs. If a rule of the plan changes, these tests say
which cases no longer cover what they are there for."""
import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_q4 import Cache, bf16
from test_gpu_q4_attn import SCALE, check, queries
from test_gpu_q4_failure import Call

pytestmark = pytest.mark.gpu


class _Node(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS, as libcuda has it."""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kernel", ctypes.c_void_p), ("context", ctypes.c_void_p)]


def kernels(fn):
    """(name, blocks, CTAs to a cluster) of each kernel that fn enqueues."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        fn()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph, stream=stream):
        fn()
    raw, cu, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.CDLL("libcuda.so.1"), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    got = []
    for node in map(ctypes.c_void_p, nodes):
        kind, p, name = ctypes.c_int(0), _Node(), ctypes.c_char_p()
        assert cu.cuGraphNodeGetType(node, ctypes.byref(kind)) == 0
        if kind.value != 0:
            continue
        assert cu.cuGraphKernelNodeGetParams_v2(node, ctypes.byref(p)) == 0
        cluster = (ctypes.c_uint * 16)()
        assert cu.cuGraphKernelNodeGetAttribute(node, 4, cluster) == 0  # cluster dimension
        assert cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)) == 0
        got.append((name.value.decode(), p.grid[0], max(1, cluster[0])))
    return got


def way_of(c, q, bound):
    """(columns / 8, CTAs to a cluster; 0: cut and merged) of a call."""
    call = Call(c, q, max_seq_len=bound)

    def fn():
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert zl.lib().zl_decode_attn_q4(ctypes.byref(call.p), stream) == zl.OK

    got = kernels(fn)
    name, blocks, cluster = got[0]
    nt, in_clusters = (2 if "Li2E" in name else 1), "Lb1E" in name
    assert "q4_decode_kernel" in name and in_clusters == (cluster > 1) and blocks % cluster == 0
    if len(got) == 2:
        assert "q4_merge_kernel" in got[1][0] and cluster == 1 and call.p.workspace_bytes > 0
        return nt, 0
    assert len(got) == 1 and call.p.workspace_bytes == 0
    return nt, cluster


def ragged(B, hi, q_len=1):
    return [hi] + [q_len + (i * 2741) % (hi - q_len + 1) for i in range(1, B)]


# lens, Hq, Hkv, query tokens, page size, and the way with a bound
WAYS = [
    # a CTA to a unit; heads side by side, and alone
    ([64, 0, 33], 8, 2, 1, 16, (1, 1)), ([64, 3, 33], 8, 2, 3, 16, (2, 1)),
    (ragged(51, 32, 5), 32, 8, 5, 16, (2, 1)), (ragged(64, 120), 32, 8, 1, 16, (1, 1)),
    (ragged(40, 90), 12, 6, 1, 16, (1, 1)), (ragged(90, 60, 2), 8, 4, 2, 16, (1, 1)),
    # clusters of 2, of 4, of 8, with 8, 4 and 2 slices
    (ragged(8, 1500), 32, 8, 1, 16, (1, 2)), (ragged(26, 1000), 12, 6, 1, 16, (1, 2)),
    (ragged(76, 500), 4, 4, 1, 32, (1, 2)), (ragged(2, 1500, 5), 32, 8, 5, 16, (2, 2)),
    (ragged(18, 1500, 5), 12, 6, 5, 48, (2, 2)),
    ([700, 0, 33, 1999], 8, 2, 1, 16, (1, 4)), ([2000, 1, 513, 257], 32, 8, 1, 48, (1, 4)),
    (ragged(13, 2000), 12, 6, 1, 16, (1, 4)), ([1500, 40], 5, 1, 3, 32, (2, 4)),
    ([1000] * 19, 8, 1, 2, 16, (2, 4)), (ragged(9, 3000, 5), 12, 6, 5, 16, (2, 4)),
    (ragged(26, 6000), 8, 1, 1, 64, (1, 8)), (ragged(9, 3000), 12, 6, 1, 16, (1, 8)),
    # cut all the same
    ([7000, 300], 8, 1, 1, 128, (1, 0)), ([4000], 32, 1, 2, 64, (2, 0)),
]


@pytest.mark.parametrize("lens,Hq,Hkv,q_len,P,way", WAYS)
def test_the_way_of_a_call_and_its_result(lens, Hq, Hkv, q_len, P, way):
    c = Cache(len(lens) + Hq + q_len, lens, Hkv, P)
    q = queries(c, q_len, Hq)
    assert way_of(c, q, max(lens)) == way
    assert way_of(c, q, 0) == (way[0], 0)  # without a bound the host cannot tell
    check(c, q, max_seq_len=max(lens))


@pytest.mark.parametrize("q_len,lens", [(1, [1900, 30, 333, 1]), (3, [1400, 30, 333, 3])])
def test_clusters_in_a_graph(q_len, lens):
    """Replayed over growing sequences with other queries and another graph in between: the
    bits of calls that are waited for."""
    Hq, Hkv, bound = 8, 2, 2000
    c = Cache(40 + q_len, [L + 6 for L in lens], Hkv)
    q = queries(c, q_len, Hq).cuda()
    assert way_of(c, q.cpu(), bound)[1] == 4
    pool, bt, sl = c.on_gpu()
    sl -= 6
    out, other = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(q.shape[:3], device="cuda")
    args = dict(page_size=c.P, scale=SCALE)

    def step():
        zl.decode_attn_q4(q, pool, bt, sl, out=out, lse=lse, max_seq_len=bound, **args)

    def cut():
        zl.decode_attn_q4(q, pool, bt, sl, out=other, **args)

    stream, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(stream):
        step()
        cut()
    stream.synchronize()
    for fn in (step, cut):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            fn()
            fn()
        graphs.append(g)
    inputs, got = [queries(c, q_len, Hq) for _ in range(6)], []
    for x in inputs:
        q.copy_(x)
        graphs[0].replay()
        got.append((out.clone(), lse.clone()))
        graphs[1].replay()
        sl += 1
    torch.cuda.synchronize()
    sl -= 6
    for x, (o, l) in zip(inputs, got):
        q.copy_(x)
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse) and bool(torch.isfinite(o).all())
        cut()
        # two cuts of the same sums: each within bf16's half step and fp16's of P
        assert torch.allclose(o.float(), other.float(), rtol=2.0 ** -6, atol=2.0 ** -8)
        sl += 1


def test_clusters_on_two_streams_at_once():
    """Calls in clusters beside others in clusters and cut ones."""
    caches = [Cache(50, [1900, 30, 333, 1], 2), Cache(51, ragged(8, 1500), 8)]
    qs = [queries(caches[0], 1, 8), queries(caches[1], 1, 32)]
    bounds = [2000, 1500]
    assert [way_of(c, q, n) for c, q, n in zip(caches, qs, bounds)] == [(1, 4), (1, 2)]
    on = [c.on_gpu() for c in caches]
    qs = [q.cuda() for q in qs]

    def attend(i, bound, stream=None):
        return zl.decode_attn_q4(qs[i], *on[i], page_size=16, scale=SCALE, max_seq_len=bound,
                                 stream=stream)

    want = [[attend(i, n) for n in (bounds[i], 0)] for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for k in range(30):
        for i, s in enumerate(streams):
            got[i].append(attend(i, 0 if k % 3 == 2 else bounds[i], s))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for k, x in enumerate(many):
            assert torch.equal(x, w[k % 3 == 2])


@pytest.mark.parametrize("way", [dict(), dict(num_ctas=3), dict(max_seq_len=600)])
@pytest.mark.parametrize("size", [1e4, 1e30])
def test_large_scores_pick_single_tokens(size, way):
    """Where the best score leads by more than the roundings of scores (plain_q4.tolerance's e)
    and 40, every other weight is below 2^-57: the row is the best token's V. That has 6
    significant bits, and what is computed lies within 2^-20 of it, so it comes out exact, but
    for the others' part: up to 600 tokens times 2^-57 (2^-47) of the largest value, which
    shows where V is 0 and vanishes in the rounding to bf16 elsewhere."""
    c = Cache(60, [600, 33, 200], 2, spread=0.5)
    q = (queries(c, 2, 8).double() * size).bfloat16()
    pool, bt, sl = c.on_gpu()
    out = bf16(zl.decode_attn_q4(q.cuda(), pool, bt, sl, page_size=c.P, scale=SCALE, **way))
    rows = 0
    for b, L in enumerate(c.lens):
        k, v = c.kv(b)
        for i in range(2):
            see = L - 1 + i
            for h in range(8):
                x = k[:see, h // 4] @ bf16(q)[b, i, h] * SCALE
                mag = (np.abs(k[:see, h // 4]) @ np.abs(bf16(q)[b, i, h])).max() * SCALE
                e = 16 * 2.0 ** -23 * mag + 3 * 2.0 ** -23 * (np.abs(x).max() + 16)
                best, second = np.argmax(x), np.sort(x)[-2]
                # (both scores off by e, and the parts' log-sum-exps by as much)
                if x[best] - second > 40 + 4 * e:
                    rows += 1
                    assert v[best, h // 4].any()
                    want, part = v[best, h // 4], 2.0 ** -47 * np.abs(v[:, h // 4]).max()
                    assert (np.abs(out[b, i, h] - want) <= np.where(want == 0, part, 0)).all()
    assert rows >= 40  # of 48
