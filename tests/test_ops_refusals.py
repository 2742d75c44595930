"""What the eviction, the commit and the weighted attention refuse on the host
beyond the plain checks of their arguments (CPU only)."""
import ctypes

import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from test_ops_abi import FAKE, _evict


def evict_status(**over):
    return zl.lib().zl_kv_evict(ctypes.byref(_evict(**over)), None)


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
