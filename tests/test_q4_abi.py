"""The entry points around the 4-bit cache refuse bad arguments on the host, before
anything reaches a GPU (CPU only)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
import plain_q4

FAKE = 1 << 20
NO_GPU = not torch.cuda.is_available()


def _fill(p, **over):
    p.struct_size = ctypes.sizeof(p)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _append(**over):
    return _fill(zl.AppendQ4Params(), **{**dict(
        k_new=FAKE, v_new=FAKE, k_stride=1024, v_stride=1024, pool=FAKE, page_stride=16 * 8 * 144,
        token_stride=8 * 144, head_stride=144, block_table=FAKE, block_table_stride=8,
        seq_lens=FAKE, B=4, q_len=2, Hkv=8, page_size=16, num_pages=64), **over})


def _read(**over):
    return _fill(zl.ReadQ4Params(), **{**dict(
        pool=FAKE, page_stride=16 * 8 * 144, token_stride=8 * 144, head_stride=144,
        block_table=FAKE, block_table_stride=8, seq_lens=FAKE, k_out=FAKE, v_out=FAKE, B=4,
        tokens=100, Hkv=8, page_size=16, num_pages=64), **over})


def _decode(**over):
    return _fill(zl.DecodeQ4Params(), **{**dict(
        q=FAKE, pool=FAKE, page_stride=16 * 8 * 144, token_stride=8 * 144, head_stride=144,
        block_table=FAKE, block_table_stride=8, seq_lens=FAKE, out=FAKE, B=4, q_len=1, Hq=32,
        Hkv=8, page_size=16, num_pages=64, scale=0.1), **over})


TURNS = (ctypes.c_uint64 * 64)()
AXES = (ctypes.c_uint8 * 64)()


def _norm(**over):
    return _fill(zl.NormRopeParams(), **{**dict(
        q=FAKE, k=2 * FAKE, v=3 * FAKE, q_stride=4096, k_stride=1024, v_stride=1024,
        q_out=4 * FAKE, k_out=5 * FAKE, q_out_stride=4096, k_out_stride=1024, eps=1e-6,
        rope_scale=1.0, freq_turns=ctypes.addressof(TURNS), axes=ctypes.addressof(AXES), n_freq=64,
        n_axes=1, cache=zl.CACHE_Q4, k_pool=6 * FAKE, page_stride=16 * 8 * 144,
        token_stride=8 * 144, head_stride=144, block_table=FAKE, block_table_stride=8,
        seq_lens=FAKE, B=4, q_len=2, Hq=32, Hkv=8, page_size=16, num_pages=64), **over})


def status(name, p):
    return getattr(zl.lib(), name)(ctypes.byref(p), None)


POOL = [
    dict(struct_size=8), dict(B=0), dict(Hkv=0), dict(page_size=0), dict(num_pages=0),
    dict(block_table_stride=0), dict(pool=None), dict(pool=FAKE + 8), dict(block_table=None),
    dict(block_table=FAKE + 2), dict(seq_lens=None), dict(seq_lens=FAKE + 1),
    dict(err_flags=FAKE + 2), dict(page_stride=0), dict(token_stride=-144),
    dict(head_stride=150), dict(token_stride=8),
]


@pytest.mark.parametrize("over", POOL + [
    dict(q_len=0), dict(k_new=None), dict(v_new=None), dict(k_new=FAKE + 8), dict(k_stride=1020),
    dict(v_stride=1016), dict(new_lens=FAKE + 2),
])
def test_append_refuses(over):
    assert status("zl_kv_append_q4", _append(**over)) == zl.ERR_INVALID_ARG


@pytest.mark.parametrize("over", POOL + [
    dict(tokens=0), dict(k_out=None, v_out=None), dict(k_out=FAKE + 16), dict(v_out=FAKE + 16),
])
def test_read_refuses(over):
    assert status("zl_kv_read_q4", _read(**over)) == zl.ERR_INVALID_ARG


@pytest.mark.parametrize("over", POOL + [
    dict(q_len=0), dict(Hq=0), dict(Hq=30), dict(q=None), dict(out=None), dict(q=FAKE + 8),
    dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=-1.0), dict(num_ctas=-1), dict(max_seq_len=-1),
])
def test_decode_refuses(over):
    assert status("zl_decode_attn_q4", _decode(**over)) == zl.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(B=4097), dict(q_len=129), dict(Hq=8 * 129), dict(page_size=24), dict(page_size=1040),
    dict(num_ctas=70000), dict(block_table_stride=1 << 40),
    dict(B=4096, block_table_stride=1 << 19),          # 2^31 tiles
    dict(Hkv=32768, Hq=32768, block_table_stride=1 << 24),
])
def test_decode_does_not_support(over):
    assert status("zl_decode_attn_q4", _decode(**over)) == zl.ERR_UNSUPPORTED
    n = ctypes.c_size_t(0)
    assert zl.lib().zl_decode_attn_q4_workspace_size(
        ctypes.byref(_decode(**over)), ctypes.byref(n)) == zl.ERR_UNSUPPORTED


def test_more_sequences_or_rows_than_a_grid_holds():
    assert status("zl_kv_append_q4", _append(B=65536)) == zl.ERR_UNSUPPORTED
    assert status("zl_kv_append_q4", _append(q_len=1 << 28)) == zl.ERR_UNSUPPORTED
    assert status("zl_kv_read_q4", _read(B=65536)) == zl.ERR_UNSUPPORTED
    assert status("zl_kv_read_q4", _read(tokens=(1 << 31) - 1)) == zl.ERR_UNSUPPORTED


@pytest.mark.parametrize("over", [
    dict(struct_size=8), dict(B=0), dict(q_len=0), dict(Hq=0), dict(Hkv=0), dict(q=None),
    dict(k=None), dict(q_out=None), dict(v=None), dict(q=FAKE + 8), dict(k_out=5 * FAKE + 2),
    dict(q_stride=4095), dict(q_stride=4088), dict(k_stride=1016), dict(q_out_stride=0),
    dict(k_out_stride=1000), dict(v_stride=0), dict(eps=-1.0), dict(eps=float("nan")),
    dict(rope_scale=float("inf")), dict(n_freq=-16), dict(n_axes=0), dict(freq_turns=None),
    dict(q_weight=FAKE + 4), dict(positions=FAKE + 2), dict(n_axes=2, positions=FAKE, axis_stride=7),
    dict(cache=3), dict(cache=-1), dict(cache=zl.CACHE_BF16), dict(v_pool=7 * FAKE),
    dict(k_pool=None), dict(k_pool=6 * FAKE + 8), dict(head_stride=8), dict(page_stride=0),
    dict(block_table=None), dict(seq_lens=None), dict(page_size=0), dict(num_pages=0),
    dict(cache=zl.CACHE_NONE, k_out=None), dict(cache=zl.CACHE_NONE, seq_lens=None),
    # written over what is read
    dict(q_out=FAKE + 16), dict(q_out=FAKE, q_out_stride=4104), dict(q_out=2 * FAKE),
    dict(k_out=3 * FAKE), dict(k_out=4 * FAKE + 256), dict(k_out=FAKE), dict(q_out=3 * FAKE - 512),
])
def test_norm_rope_refuses(over):
    assert status("zl_qk_norm_rope", _norm(**over)) == zl.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(n_freq=8), dict(n_freq=65), dict(n_freq=80), dict(n_axes=5),
    dict(Hq=65536, q_stride=1 << 24, q_out_stride=1 << 24, q=1 << 40, q_out=1 << 41),
])
def test_norm_rope_does_not_support(over):
    assert status("zl_qk_norm_rope", _norm(**over)) == zl.ERR_UNSUPPORTED


def test_an_axis_out_of_range():
    axes = (ctypes.c_uint8 * 64)(*([0] * 63 + [2]))
    over = dict(axes=ctypes.addressof(axes), n_axes=2, positions=FAKE, axis_stride=8)
    assert status("zl_qk_norm_rope", _norm(**over)) == zl.ERR_INVALID_ARG


@pytest.mark.skipif(not NO_GPU, reason="a GPU is present")
def test_valid_calls_reach_the_device():
    for name, p in (("zl_kv_append_q4", _append()), ("zl_kv_read_q4", _read(v_out=None)),
                    ("zl_decode_attn_q4", _decode()), ("zl_qk_norm_rope", _norm()),
                    # rows interleaved in one buffer of [token][q | k | v], in place
                    ("zl_qk_norm_rope", _norm(q=FAKE, k=FAKE + 8192, v=FAKE + 10240, q_out=FAKE,
                                              k_out=FAKE + 8192, q_stride=6144, k_stride=6144,
                                              v_stride=6144, q_out_stride=6144,
                                              k_out_stride=6144)),
                    ("zl_qk_norm_rope", _norm(n_freq=0, freq_turns=None, axes=None,
                                              cache=zl.CACHE_NONE, seq_lens=None, v=None))):
        assert status(name, p) == zl.ERR_CUDA


def test_null_params():
    for name in ("zl_kv_append_q4", "zl_kv_read_q4", "zl_decode_attn_q4", "zl_qk_norm_rope"):
        assert getattr(zl.lib(), name)(None, None) == zl.ERR_INVALID_ARG
    assert zl.lib().zl_decode_attn_q4_workspace_size(ctypes.byref(_decode()),
                                                     None) == zl.ERR_INVALID_ARG


@pytest.mark.parametrize("form,mirror", [
    ("_APPEND_Q4", "AppendQ4Params"), ("_READ_Q4", "ReadQ4Params"),
    ("_DECODE_Q4", "DecodeQ4Params"), ("_NORM_ROPE", "NormRopeParams")])
def test_packed_structs_match_the_mirrors(form, mirror):
    form, mirror = getattr(zl, form), getattr(zl, mirror)
    n = len(mirror._fields_)
    got = mirror.from_buffer_copy(form.pack(*range(1, n + 1)))
    assert [float(getattr(got, name) or 0) for name, _ in mirror._fields_] == list(range(1, n + 1))


def test_constants_match_the_header():
    text = open(zl.HEADER).read()
    assert f"#define ZL_Q4_ROW_BYTES {zl.Q4_ROW_BYTES}" in text
    for name, value in (("NONE", zl.CACHE_NONE), ("BF16", zl.CACHE_BF16), ("Q4", zl.CACHE_Q4)):
        assert f"ZL_CACHE_{name} = {value}" in text


# ------------------------------------------------------------------- rotations
def test_turns_of_a_rope():
    """Frequencies in turns per position, 64 bits behind the point."""
    freq = [1.0, 0.0, -1.0, 1e-9, 6.283185307179586, 1000.0] + [0.5] * 10
    r = zl.Rope(freq)
    turns = list(r._turns)
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937511")
    for f, t in zip(freq, turns):
        exact = Fraction(f) / two_pi
        gap = (Fraction(t, 1 << 64) - exact) % 1
        assert min(gap, 1 - gap) <= Fraction(1, 1 << 65)
    assert (turns[0] + turns[2]) % (1 << 64) == 0
    assert zl.rope_frequencies(64, 10000.0)[:2] == [1.0, 10000.0 ** (-2 / 64)]
    assert len(zl.rope_frequencies(64)) == 32


def test_rope_refuses():
    for kw in (dict(frequencies=[float("nan")] * 16), dict(frequencies=[1.0] * 16, axes=[0] * 15),
               dict(frequencies=[1.0] * 16, axes=[4] * 16),
               dict(frequencies=[1.0] * 16, axes=[-1] * 16)):
        with pytest.raises(ValueError):
            zl.Rope(**kw)


# --------------------------------------------------------- the binding's checks
def _tensors(B=2, q_len=3, Hq=8, Hkv=2, P=16, pages=6):
    rows = lambda h: torch.zeros(B, q_len, h, 128, dtype=torch.bfloat16)  # noqa: E731
    return dict(q=rows(Hq), k=rows(Hkv), v=rows(Hkv),
                pool=torch.zeros(pages, P, Hkv, 144, dtype=torch.uint8),
                kp=torch.zeros(pages, P, Hkv, 128, dtype=torch.bfloat16),
                bt=torch.zeros(B, 3, dtype=torch.int32), sl=torch.ones(B, dtype=torch.int32))


def test_calls_off_the_gpu_are_refused():
    d = _tensors()
    at = dict(page_size=16)
    for call in (lambda: zl.decode_attn_q4(d["q"], d["pool"], d["bt"], d["sl"], scale=0.1, **at),
                 lambda: zl.kv_append_q4(d["k"], d["v"], d["pool"], d["bt"], d["sl"], **at),
                 lambda: zl.kv_read_q4(d["pool"], d["bt"], d["sl"], tokens=9, **at),
                 lambda: zl.qk_norm_rope(d["q"], d["k"])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("change", [
    dict(pool=torch.zeros(6, 16, 2, 144, dtype=torch.int8)),
    dict(pool=torch.zeros(6, 16, 2, 128, dtype=torch.uint8)),
    dict(pool=torch.zeros(6, 16, 288, dtype=torch.uint8)),
    dict(pool=torch.zeros(6, 32, 2, 144, dtype=torch.uint8)),
    dict(pool=torch.zeros(6, 16, 2, 288, dtype=torch.uint8)[..., ::2]),
    dict(sl=torch.ones(2, dtype=torch.int64)), dict(sl=torch.ones(3, dtype=torch.int32)),
    dict(bt=torch.zeros(2, 3, dtype=torch.int64)), dict(bt=torch.zeros(6, dtype=torch.int32)),
    dict(bt=torch.zeros(1, 3, dtype=torch.int32).expand(2, 3)),
    dict(q=torch.zeros(2, 3, 8, 128)), dict(q=torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16)),
    dict(q=torch.zeros(3, 3, 8, 128, dtype=torch.bfloat16)),
    dict(layout="NDH"), dict(out=torch.zeros(2, 3, 8, 128)), dict(lse=torch.zeros(2, 3)),
    dict(err_flags=torch.zeros(1)),
])
def test_decode_refuses_wrong_tensors(change):
    d = {**_tensors(), **change}
    kw = {n: d[n] for n in ("layout", "out", "lse", "err_flags") if n in d}
    with pytest.raises(ValueError) as e:
        zl.decode_attn_q4(d["q"], d["pool"], d["bt"], d["sl"], page_size=16, scale=0.1, **kw)
    assert "CUDA" not in str(e.value)


@pytest.mark.parametrize("change", [
    dict(k=torch.zeros(2, 3, 2, 128)), dict(k=torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)),
    dict(v=torch.zeros(2, 2, 2, 128, dtype=torch.bfloat16)),
    dict(k=torch.zeros(2, 3, 256, dtype=torch.bfloat16)),
    dict(k=torch.zeros(2, 3, 2, 256, dtype=torch.bfloat16)[..., ::2]),
    dict(k=torch.zeros(2, 2, 3, 128, dtype=torch.bfloat16).transpose(1, 2)),
    dict(k=torch.zeros(2, 6, 2, 128, dtype=torch.bfloat16)[:, ::2][:, :, ::1].flip(0)[:, :2]),
    dict(v=torch.zeros(2, 5, 2, 128, dtype=torch.bfloat16)[:, :3]),  # not evenly spaced
    dict(new_lens=torch.zeros(3, dtype=torch.int32)), dict(new_lens=torch.zeros(2)),
])
def test_append_refuses_wrong_tensors(change):
    d = {**_tensors(), **change}
    with pytest.raises(ValueError) as e:
        zl.kv_append_q4(d["k"], d["v"], d["pool"], d["bt"], d["sl"], page_size=16,
                        new_lens=d.get("new_lens"))
    assert "CUDA" not in str(e.value)


@pytest.mark.parametrize("kw", [
    dict(), dict(tokens=0), dict(k_out=torch.zeros(2, 9, 2, 128)),
    dict(k_out=torch.zeros(2, 9, 2, 128, dtype=torch.bfloat16), tokens=8),
    dict(k_out=torch.zeros(2, 9, 3, 128, dtype=torch.bfloat16)),
    dict(k_out=torch.zeros(2, 9, 2, 128, dtype=torch.bfloat16),
         v_out=torch.zeros(2, 8, 2, 128, dtype=torch.bfloat16)),
    dict(v_out=torch.zeros(2, 9, 256, dtype=torch.bfloat16)),
])
def test_read_refuses_wrong_tensors(kw):
    d = _tensors()
    with pytest.raises(ValueError):
        zl.kv_read_q4(d["pool"], d["bt"], d["sl"], page_size=16, **kw)


@pytest.mark.parametrize("kw", [
    dict(rope=zl.Rope([1.0] * 16)),                                   # no positions
    dict(rope=zl.Rope([1.0] * 16), positions=torch.zeros(2, 3)),
    dict(rope=zl.Rope([1.0] * 16), positions=torch.zeros(2, 4, dtype=torch.int32)),
    dict(rope=zl.Rope([1.0] * 16, axes=[1] * 16), positions=torch.zeros(2, 3, dtype=torch.int32)),
    dict(rope=zl.Rope([1.0] * 16, axes=[2] * 16),
         positions=torch.zeros(2, 2, 3, dtype=torch.int32)),
    dict(q_weight=torch.ones(64)), dict(k_weight=torch.ones(128, dtype=torch.bfloat16)),
    dict(q_out=torch.zeros(2, 3, 7, 128, dtype=torch.bfloat16)),
    dict(k_out=torch.zeros(2, 3, 2, 128)), dict(pool="pool"), dict(pool="pool", v="v"),
    dict(pool="pool", v="v", block_table="bt"), dict(k_pool="kp", v="v"),
    dict(pool="pool", k_pool="kp", v_pool="kp"),
    dict(pool="pool", v="v", block_table="bt", seq_lens="sl", page_size=32),
    dict(pool="kp", v="v", block_table="bt", seq_lens="sl", page_size=16),
    dict(k_pool="pool", v_pool="pool", v="v", block_table="bt", seq_lens="sl", page_size=16),
    dict(pool="pool", v=torch.zeros(2, 3, 1, 128, dtype=torch.bfloat16), block_table="bt",
         seq_lens="sl", page_size=16),
    dict(pool="pool", v="v", block_table=torch.zeros(3, 3, dtype=torch.int32),
         seq_lens=torch.ones(3, dtype=torch.int32), page_size=16),
])
def test_norm_rope_refuses_wrong_tensors(kw):
    d = _tensors()
    kw = {n: d[x] if isinstance(x, str) else x for n, x in kw.items()}
    with pytest.raises(ValueError) as e:
        zl.qk_norm_rope(d["q"], d["k"], **kw)
    assert "CUDA" not in str(e.value)


# ------------------------------------------------------------- the plain forms
def test_the_plain_quantisation_on_known_blocks():
    x = np.zeros((4, 128))
    x[0, :8] = [6, -6, 5, 2.5, 0.25, 0.75, -3.5, 1.25]      # scale 1: every tie
    x[1, 0] = 61440.0                                        # the largest scale
    x[1, 16] = 1e30                                          # beyond it
    x[2, 0] = 6 * 2.0 ** -18                                 # rounds to scale 0
    x[3, 0], x[3, 1] = 6 * 1.0625, 3.0                       # 1.0625 is a tie: 1
    code, byte = plain_q4.quantise(x)
    assert code[0, :8].tolist() == [7, 15, 6, 4, 0, 2, 14, 2]
    assert byte[0, 0] == 15 << 3 and byte[1, 0] == byte[1, 1] == plain_q4.TOP and code[1, 16] == 7
    assert byte[2, 0] == 0 and code[2, 0] == 0 and byte[3, 0] == 15 << 3
    k, v = plain_q4.unpack(plain_q4.pack(x, -x))
    assert k[0, :8].tolist() == [6, -6, 4, 2, 0, 1, -4, 1] and (v == -k).all()
    # a value of an exact grid comes back as it is
    assert (plain_q4.unpack(plain_q4.pack(k, v))[0] == k).all()


# ------------------------------------------------------------ copies of a rotation
def _handed_over(monkeypatch, rope):
    """The parameters that a norm call with this rope hands to the library (a fake one)."""
    import contextlib
    got = []

    def entry(packed, stream):
        got.append(zl.NormRopeParams.from_buffer_copy(packed))
        return zl.OK

    monkeypatch.setattr(zl, "_on", lambda index, stream: (0, contextlib.nullcontext()))
    monkeypatch.setitem(zl._raw, "zl_qk_norm_rope", entry)
    d = _tensors()
    zl.qk_norm_rope(d["q"], d["k"], rope=rope, positions=torch.zeros(4, 2, 3, dtype=torch.int32))
    return got[0]


@pytest.mark.parametrize("how", ["itself", "copy", "deepcopy", "pickle", "subclass"])
def test_a_copied_rope_hands_over_its_own_arrays(monkeypatch, how):
    """Whatever becomes of the original: its arrays are freed with it."""
    import copy
    import pickle

    freq, axes = [0.5, 1.0, -2.0, 3.0] * 8, [0, 1, 2, 3] * 8
    make = zl.Rope if how != "subclass" else type("Own", (zl.Rope,), {})
    first = make(freq, axes=axes, interleaved=True, scale=1.5)
    first.note = [1]
    rope = {"itself": lambda: first, "copy": lambda: copy.copy(first),
            "deepcopy": lambda: copy.deepcopy(first), "subclass": lambda: copy.deepcopy(first),
            "pickle": lambda: pickle.loads(pickle.dumps(first))}[how]()
    assert type(rope) is type(first) and rope.note == [1]
    p = _handed_over(monkeypatch, rope)
    assert p.freq_turns == ctypes.addressof(rope._turns) and p.axes == ctypes.addressof(rope._axes)
    assert (p.n_freq, p.n_axes, p.interleaved, p.rope_scale) == (32, 4, 1, 1.5)
    assert list(rope._turns) == list(first._turns) and list(rope._axes) == axes
    if rope is not first:
        assert p.freq_turns != ctypes.addressof(first._turns)


def test_a_rope_inside_a_copied_model(monkeypatch):
    import copy
    model = {"layers": [zl.Rope(zl.rope_frequencies(64))]}
    twin = copy.deepcopy(model)
    want = list(model["layers"][0]._turns)
    del model
    rope = twin["layers"][0]
    p = _handed_over(monkeypatch, rope)
    assert p.freq_turns == ctypes.addressof(rope._turns) and list(rope._turns) == want


@pytest.mark.parametrize("flags", [1, 0x40000000, 0x80000001])
def test_decode_refuses_flags_that_are_none(flags):
    assert status("zl_decode_attn_q4", _decode(flags=flags)) == zl.ERR_INVALID_ARG
    if NO_GPU:
        assert status("zl_decode_attn_q4", _decode(flags=zl.TEST_STALL)) == zl.ERR_CUDA
