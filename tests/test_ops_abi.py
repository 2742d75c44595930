"""The entry points for modified scores, eviction and path commit refuse bad
arguments on the host, before anything reaches a GPU (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from plain_ops import mask_bits
from test_abi import _params

FAKE = 1 << 20


def _scores(**over):
    m = zl.ScoreParams()
    m.struct_size = ctypes.sizeof(zl.ScoreParams)
    m.weights_decay = 1.0
    m.weights_tokens, m.weights_head_stride, m.weights_seq_stride = 128, 128, 8 * 128
    for k, v in over.items():
        setattr(m, k, v)
    return m


@pytest.mark.parametrize("over,mods,code", [
    (dict(), dict(struct_size=8), zl.ERR_INVALID_ARG),
    (dict(), dict(softcap=-1.0), zl.ERR_INVALID_ARG),
    (dict(), dict(softcap=float("nan")), zl.ERR_INVALID_ARG),
    (dict(), dict(softcap=float("inf")), zl.ERR_INVALID_ARG),
    (dict(), dict(softcap=1e-30), zl.ERR_UNSUPPORTED),
    (dict(), dict(softcap=1e30), zl.ERR_UNSUPPORTED),
    (dict(), dict(window=-1), zl.ERR_INVALID_ARG),
    (dict(), dict(alibi_slopes=FAKE + 2), zl.ERR_INVALID_ARG),
    (dict(), dict(tree_mask=FAKE + 1), zl.ERR_INVALID_ARG),
    (dict(), dict(weights=FAKE + 2), zl.ERR_INVALID_ARG),
    (dict(), dict(weights=FAKE, weights_tokens=0), zl.ERR_INVALID_ARG),
    (dict(), dict(weights=FAKE, weights_decay=-0.5), zl.ERR_INVALID_ARG),
    (dict(), dict(weights=FAKE, weights_decay=float("nan")), zl.ERR_INVALID_ARG),
    (dict(), dict(weights=FAKE, weights_head_stride=127), zl.ERR_INVALID_ARG),  # rows overlap
    (dict(), dict(weights=FAKE, weights_seq_stride=0), zl.ERR_INVALID_ARG),
    # each stride holds a row, yet (sequence 0, head 1) and (1, 0) are the same
    (dict(), dict(weights=FAKE, weights_head_stride=256, weights_seq_stride=256),
     zl.ERR_INVALID_ARG),
    (dict(), dict(weights=FAKE, weights_head_stride=128, weights_seq_stride=1023),
     zl.ERR_INVALID_ARG),
    (dict(scale=1e35), dict(softcap=1e-6), zl.ERR_UNSUPPORTED),  # scale / softcap overflows
    (dict(scale=1e-35), dict(softcap=1e6), zl.ERR_UNSUPPORTED),
    (dict(flags=zl.SINGLE_LAUNCH), dict(softcap=30.0), zl.ERR_UNSUPPORTED),
    (dict(flags=zl.TEST_STALL), dict(), zl.ERR_UNSUPPORTED),
    (dict(shared_prefix_pages=1), dict(softcap=30.0), zl.ERR_UNSUPPORTED),
    (dict(q=None), dict(softcap=30.0), zl.ERR_INVALID_ARG),
    (dict(D_qk=64, D_v=64), dict(softcap=30.0), zl.ERR_UNSUPPORTED),
    (dict(page_size=8), dict(softcap=30.0), zl.ERR_UNSUPPORTED),
    (dict(k_new=FAKE), dict(softcap=30.0), zl.ERR_INVALID_ARG),
])
def test_modified_scores_host_validation(over, mods, code):
    p, m = _params(**over), _scores(**mods)
    assert zl.lib().zl_decode_attn_ex(ctypes.byref(p), ctypes.byref(m), None) == code


def test_modified_scores_null_params():
    p, m = _params(), _scores()
    n = ctypes.c_size_t(0)
    assert zl.lib().zl_decode_attn_ex(None, ctypes.byref(m), None) == zl.ERR_INVALID_ARG
    assert zl.lib().zl_decode_attn_ex(ctypes.byref(p), None, None) == zl.ERR_INVALID_ARG
    size = zl.lib().zl_decode_attn_ex_workspace_size
    assert size(ctypes.byref(p), None, ctypes.byref(n)) == zl.ERR_INVALID_ARG
    assert size(ctypes.byref(p), ctypes.byref(m), None) == zl.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert zl.lib().zl_decode_attn_ex(ctypes.byref(p), ctypes.byref(m), None) != zl.OK


def _evict(**over):
    p = zl.EvictParams()
    p.struct_size = ctypes.sizeof(zl.EvictParams)
    p.k_pool = p.v_pool = p.block_table = p.seq_lens = p.kept = p.weights = FAKE
    p.new_lens = 2 * FAKE
    p.page_stride, p.token_stride, p.head_stride = 16 * 8 * 128, 8 * 128, 128
    p.block_table_stride = 8
    p.weights_tokens, p.weights_head_stride, p.weights_seq_stride = 128, 128, 8 * 128
    p.B, p.Hkv, p.D_k, p.D_v, p.page_size, p.num_pages = 4, 8, 128, 128, 16, 64
    p.budget, p.sink, p.recent = 32, 4, 8
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over", [
    dict(struct_size=8), dict(B=0), dict(Hkv=0), dict(page_size=0), dict(num_pages=0),
    dict(block_table_stride=0), dict(D_k=12), dict(D_k=2048), dict(D_v=4),
    dict(k_pool=None), dict(block_table=None), dict(seq_lens=None), dict(new_lens=None),
    dict(kept=None), dict(weights=None), dict(k_pool=FAKE + 8), dict(weights=FAKE + 2),
    dict(token_stride=100), dict(head_stride=0), dict(budget=0), dict(sink=-1),
    dict(recent=-1), dict(sink=25),               # sink + recent > budget
    dict(sink=1 << 30, recent=1 << 30, budget=1 << 30),
    dict(weights_tokens=0), dict(weights_head_stride=100), dict(weights_seq_stride=0),
    dict(weights_head_stride=256, weights_seq_stride=256),       # rows overlap
    dict(weights_out=2 * FAKE, weights_out_head_stride=32, weights_out_seq_stride=40),
    dict(weights_out=FAKE, weights_out_head_stride=128, weights_out_seq_stride=1024),  # in place
    dict(dst_block_table=FAKE, dst_block_table_stride=8),
    dict(weights_out=FAKE, weights_out_head_stride=8, weights_out_seq_stride=1024),
    dict(weights_out=FAKE, weights_out_head_stride=32, weights_out_seq_stride=0),
    dict(dst_block_table=FAKE, dst_block_table_stride=0),
    dict(new_lens=FAKE), dict(new_lens=FAKE + 12),   # overlaps seq_lens
])
def test_evict_host_validation(over):
    p = _evict(**over)
    assert zl.lib().zl_kv_evict(ctypes.byref(p), None) == zl.ERR_INVALID_ARG


def _commit(**over):
    p = zl.CommitParams()
    p.struct_size = ctypes.sizeof(zl.CommitParams)
    p.k_pool = p.v_pool = p.block_table = p.seq_lens = p.path = p.accepted = FAKE
    p.new_lens = 2 * FAKE
    p.page_stride, p.token_stride, p.head_stride = 16 * 8 * 128, 8 * 128, 128
    p.block_table_stride, p.path_stride, p.path_len = 8, 8, 8
    p.B, p.q_len, p.Hkv, p.D_k, p.D_v, p.page_size, p.num_pages = 4, 8, 8, 128, 128, 16, 64
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code", [
    (dict(struct_size=8), zl.ERR_INVALID_ARG), (dict(B=0), zl.ERR_INVALID_ARG),
    (dict(q_len=0), zl.ERR_INVALID_ARG), (dict(q_len=129), zl.ERR_UNSUPPORTED),
    (dict(path=None), zl.ERR_INVALID_ARG), (dict(accepted=None), zl.ERR_INVALID_ARG),
    (dict(path=FAKE + 2), zl.ERR_INVALID_ARG), (dict(path_len=0), zl.ERR_INVALID_ARG),
    (dict(path_stride=4), zl.ERR_INVALID_ARG), (dict(new_lens=FAKE + 4), zl.ERR_INVALID_ARG),
    (dict(D_k=1032), zl.ERR_INVALID_ARG), (dict(k_pool=FAKE + 8), zl.ERR_INVALID_ARG),
    (dict(B=70000, new_lens=1 << 24), zl.ERR_UNSUPPORTED),
])
def test_commit_host_validation(over, code):
    p = _commit(**over)
    assert zl.lib().zl_kv_commit(ctypes.byref(p), None) == code


def test_null_params_and_no_cpu_fallback():
    assert zl.lib().zl_kv_evict(None, None) == zl.ERR_INVALID_ARG
    assert zl.lib().zl_kv_commit(None, None) == zl.ERR_INVALID_ARG
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for fn, p in ((zl.lib().zl_kv_evict, _evict()), (zl.lib().zl_kv_commit, _commit())):
        assert fn(ctypes.byref(p), None) == zl.ERR_CUDA


def test_bad_path_bit_matches_the_header():
    assert f"#define ZL_DEVERR_BAD_PATH {zl.DEVERR_BAD_PATH}u" in open(zl.HEADER).read()


@pytest.mark.parametrize("form,mirror", [("_PARAMS", "Params"), ("_SCORES", "ScoreParams"),
                                         ("_EVICT", "EvictParams"), ("_COMMIT", "CommitParams")])
def test_packed_structs_match_the_mirrors(form, mirror):
    """The binding packs the parameter structs in one step: every field where
    the ctypes mirror has it."""
    form, mirror = getattr(zl, form), getattr(zl, mirror)
    n = len(mirror._fields_)
    got = mirror.from_buffer_copy(form.pack(*range(1, n + 1)))
    assert [float(getattr(got, name)) for name, _ in mirror._fields_] == list(range(1, n + 1))


# ------------------------------------------------------------ the binding's checks
def _tensors(B=2, q_len=3, Hq=8, Hkv=2, P=16, pages=6):
    return dict(q=torch.zeros(B, q_len, Hq, 128, dtype=torch.bfloat16),
                k=torch.zeros(pages, P, Hkv, 128, dtype=torch.bfloat16),
                v=torch.zeros(pages, P, Hkv, 128, dtype=torch.bfloat16),
                bt=torch.zeros(B, 3, dtype=torch.int32), sl=torch.ones(B, dtype=torch.int32))


@pytest.mark.parametrize("mods", [
    dict(alibi_slopes=torch.zeros(7)), dict(alibi_slopes=torch.zeros(8, dtype=torch.float64)),
    dict(tree_mask=torch.zeros(2, 3, 1)), dict(tree_mask=torch.zeros(2, 3, 2, dtype=torch.int32)),
    dict(tree_mask=torch.zeros(2, 2, 1, dtype=torch.int32)),
    dict(weights=torch.zeros(2, 8, 48)), dict(weights=torch.zeros(2, 2, 48, dtype=torch.float64)),
    dict(weights=torch.zeros(2, 2, 48, 1)), dict(weights=torch.zeros(2, 2, 96)[:, :, ::2]),
])
def test_decode_attn_refuses_wrong_tensors(mods):
    d = _tensors()
    with pytest.raises(ValueError):
        zl.decode_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], page_size=16, scale=0.1, **mods)


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(2, 3, 8, 128)), dict(sl=torch.ones(2, dtype=torch.int64)),
    dict(sl=torch.ones(3, dtype=torch.int32)), dict(bt=torch.zeros(2, 3, dtype=torch.int64)),
    dict(bt=torch.zeros(1, 3, dtype=torch.int32).expand(2, 3)),
    dict(v=torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16)),
    dict(k=torch.zeros(6, 32, 2, 128, dtype=torch.bfloat16)),
])
def test_decode_attn_with_mods_refuses_wrong_inputs(change):
    d = {**_tensors(), **change}
    with pytest.raises(ValueError):
        zl.decode_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], page_size=16, scale=0.1,
                       softcap=30.0)


def test_decode_attn_with_mods_refuses_other_modes():
    d = _tensors()
    for kw in (dict(single_launch=True), dict(shared_prefix_pages=1)):
        with pytest.raises(zl.ZlError) as e:
            zl.decode_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], page_size=16, scale=0.1,
                           window=8, **kw)
        assert e.value.status == zl.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(window=2.5), dict(window=1 << 40), dict(softcap=3.0,
                                                                             num_ctas=1 << 33)])
def test_decode_attn_refuses_numbers_out_of_range(kw):
    d = _tensors()
    with pytest.raises(ValueError):
        zl.decode_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], page_size=16, scale=0.1, **kw)


def test_calls_off_the_gpu_are_refused():
    d = _tensors()
    w = torch.zeros(2, 2, 48)
    path, acc = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for call in (lambda: zl.decode_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], page_size=16,
                                        scale=0.1, softcap=3.0),
                 lambda: zl.kv_evict(d["k"], d["v"], d["bt"], d["sl"], w, page_size=16, budget=8),
                 lambda: zl.kv_commit(d["k"], d["v"], d["bt"], d["sl"], path, acc, page_size=16,
                                      q_len=3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_evict_and_commit_refuse_wrong_tensors():
    d = _tensors()
    w = torch.zeros(2, 2, 48)

    def evict(**kw):
        a = {**dict(k=d["k"], v=d["v"], bt=d["bt"], sl=d["sl"], w=w, budget=16), **kw}
        more = {n: a[n] for n in ("kept", "weights_out", "new_lens", "dst_block_table") if n in a}
        zl.kv_evict(a["k"], a["v"], a["bt"], a["sl"], a["w"], page_size=16, budget=a["budget"],
                    **more)

    for kw in (dict(w=None), dict(w=w.double()), dict(w=torch.zeros(2, 1, 48)),
               dict(kept=torch.zeros(2, 2, 8, dtype=torch.int32)),
               dict(weights_out=torch.zeros(2, 2, 8)), dict(weights_out=torch.zeros(2, 2)),
               dict(new_lens=torch.zeros(2)), dict(sl=d["sl"].long()),
               dict(dst_block_table=torch.zeros(3, 3, dtype=torch.int32)),
               dict(k=d["k"].float())):
        with pytest.raises(ValueError):
            evict(**kw)
    path, acc = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for a, b in ((path.long(), acc), (path, acc.long()), (path[:1], acc), (path[0], acc),
                 (path, acc[:1])):
        with pytest.raises(ValueError):
            zl.kv_commit(d["k"], d["v"], d["bt"], d["sl"], a, b, page_size=16, q_len=3)


# ------------------------------------------------------------------ tree masks
@pytest.mark.parametrize("q_len", [1, 2, 31, 32, 33, 64, 100, 128])
def test_tree_mask_is_the_ancestors(q_len):
    g = np.random.default_rng(q_len)
    par = np.array([[-1 if i == 0 else int(g.integers(-1, i)) for i in range(q_len)]
                    for _ in range(3)])
    m = zl.tree_mask(par)
    assert m.dtype == torch.int32 and m.shape == (3, q_len, (q_len + 31) // 32)
    want = np.zeros((3, q_len, q_len), dtype=bool)
    for b in range(3):
        for i in range(q_len):
            j = i
            while j >= 0:
                want[b, i, j] = True
                j = par[b, j]
    assert (mask_bits(m, q_len) == want).all()


def test_tree_mask_refuses():
    for bad in ([[0]], [[-1, 1]], [[-2]], [-1, 0], [[0.5]]):
        with pytest.raises(ValueError):
            zl.tree_mask(bad)
