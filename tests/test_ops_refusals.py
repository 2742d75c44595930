"""What the eviction, the commit and the weighted attention refuse on the host
beyond the plain checks of their arguments (CPU only)."""
import ctypes

import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from test_abi import _params
from test_ops_abi import FAKE, _commit, _evict, _scores


def evict_status(**over):
    return zl.lib().zl_kv_evict(ctypes.byref(_evict(**over)), None)


def commit_status(**over):
    return zl.lib().zl_kv_commit(ctypes.byref(_commit(**over)), None)


def test_rows_to_clear():
    out = dict(weights_out=2 * FAKE, weights_out_head_stride=48, weights_out_seq_stride=8 * 48)
    assert evict_status(weights_clear=-1) == zl.ERR_INVALID_ARG
    assert evict_status(weights_clear=31, **out) == zl.ERR_INVALID_ARG   # the budget is 32
    assert evict_status(weights_clear=49, **out) == zl.ERR_INVALID_ARG   # rows overlap


def test_evict_struct_sizes():
    """Only the present size and the one before weights_clear are taken."""
    new, old = ctypes.sizeof(zl.EvictParams), zl.EvictParams.weights_clear.offset
    assert old < new
    for size in (old - 8, old + 4, new + 8):
        assert evict_status(struct_size=size) == zl.ERR_INVALID_ARG
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for size in (old, new):
        assert evict_status(struct_size=size) == zl.ERR_CUDA


@pytest.mark.parametrize("over", [
    dict(weights=FAKE + 2), dict(weights_tokens=0), dict(weights_head_stride=127),
    dict(weights_seq_stride=0), dict(weights_seq_stride=1023),
])
def test_weights_of_a_commit(over):
    rows = dict(weights=4 * FAKE, weights_tokens=128, weights_head_stride=128,
                weights_seq_stride=1024)
    assert commit_status(**{**rows, **over}) == zl.ERR_INVALID_ARG


def test_commit_struct_sizes():
    new, old = ctypes.sizeof(zl.CommitParams), zl.CommitParams.weights.offset
    for size in (old - 8, old + 8, new + 8):
        assert commit_status(struct_size=size) == zl.ERR_INVALID_ARG
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for size in (old, new):
        assert commit_status(struct_size=size) == zl.ERR_CUDA


def test_binding_checks_the_weights_of_a_commit():
    k = torch.zeros(6, 16, 2, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    path, acc = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for w in (torch.zeros(2, 8, 48), torch.zeros(2, 2, 48, dtype=torch.float64),
              torch.zeros(2, 48), torch.zeros(2, 2, 96)[:, :, ::2]):
        with pytest.raises(ValueError, match="weights"):
            zl.kv_commit(k, k, bt, sl, path, acc, page_size=16, q_len=3, weights=w)


@pytest.mark.parametrize("at", [0, 4, 12, -12])
def test_new_lengths_over_an_input_of_the_commit(at):
    """The lengths of 4 sequences written where accepted, or a row of the path, is
    still read; beside them they are taken."""
    free = dict(seq_lens=2 * FAKE, path=4 * FAKE, accepted=6 * FAKE)
    assert commit_status(**free, new_lens=6 * FAKE + at) == zl.ERR_INVALID_ARG
    assert commit_status(**free, new_lens=4 * FAKE + at) == zl.ERR_INVALID_ARG
    # rows of 8 entries, 8 apart: the last one ends 128 bytes in
    assert commit_status(**free, new_lens=4 * FAKE + 124) == zl.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        for new in (6 * FAKE + 16, 6 * FAKE - 16, 4 * FAKE + 128, 4 * FAKE - 16):
            assert commit_status(**free, new_lens=new) == zl.ERR_CUDA


def test_new_lengths_over_the_kept_list():
    free, size = dict(seq_lens=2 * FAKE, kept=4 * FAKE), 4 * 8 * 32 * 4
    for new in (4 * FAKE, 4 * FAKE - 12, 4 * FAKE + size - 4):
        assert evict_status(**free, new_lens=new) == zl.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        for new in (4 * FAKE - 16, 4 * FAKE + size):
            assert evict_status(**free, new_lens=new) == zl.ERR_CUDA


@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 8192, (1 << 31) - 16384])
def test_lengths_near_the_32_bit_limit(n):
    """The kernels count rows in 32 bits and go up to a pass beyond the last one."""
    rows = dict(weights_tokens=n, weights_head_stride=1 << 31, weights_seq_stride=1 << 34)
    out = dict(weights_out=1 << 30, weights_out_head_stride=1 << 31,
               weights_out_seq_stride=1 << 34)
    assert evict_status(budget=n, new_lens=1 << 50) == zl.ERR_UNSUPPORTED
    assert evict_status(**rows) == zl.ERR_UNSUPPORTED
    assert evict_status(weights_clear=n, **out) == zl.ERR_UNSUPPORTED


def test_weights_beyond_the_grid_that_sums_them():
    """Refused before the attention is enqueued, not after it."""
    for n, Hkv in (((1 << 31) - 1, 8), ((1 << 31) - 4096, 8), (128, 65536)):
        p = _params(Hkv=Hkv, Hq=Hkv)
        m = _scores(weights=FAKE, weights_tokens=n, weights_head_stride=1 << 32,
                    weights_seq_stride=1 << 50)
        size = ctypes.c_size_t(0)
        assert zl.lib().zl_decode_attn_ex(ctypes.byref(p), ctypes.byref(m),
                                          None) == zl.ERR_UNSUPPORTED
        assert zl.lib().zl_decode_attn_ex_workspace_size(
            ctypes.byref(p), ctypes.byref(m), ctypes.byref(size)) == zl.ERR_UNSUPPORTED
