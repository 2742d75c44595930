"""The fused append of calls with modified scores reports what it could not
store, also where no query token looks at it."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from paged_decode_attention_gqa_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_len", [3, 24])
def test_an_unseen_drafted_token_on_a_bad_page(q_len):
    """A tree whose last token nobody sees, not even itself, at the start of an
    unmapped page: its row is lost and flagged, the others are stored. A
    sequence with fewer tokens than drafted, or none, is no error."""
    w = wl.random_case(3600, B=4, Hq=8, Hkv=2, q_len=q_len, poison=False,
                       lens=[129, 200, q_len - 1, 0])
    bt = w.block_table.copy()
    bt[0, 8] = -1                                  # token 128, the last one
    mask = zl.tree_mask([[-1] + list(range(q_len - 1))] * 4)
    mask[0, q_len - 1] = 0
    kn, vn = wl.new_token_rows(3600, 4, q_len, 2, 128, 128)
    got = []
    for fused in (False, True):
        k, v, err = w.k_pool.cuda(), w.v_pool.cuda(), torch.zeros(1, dtype=torch.int32).cuda()
        btd, sl = torch.from_numpy(bt).cuda(), torch.from_numpy(w.seq_lens).cuda()
        new = dict(k_new=kn.cuda(), v_new=vn.cuda())
        if not fused:
            zl.kv_append(*new.values(), k, v, btd, sl, page_size=16)
            new = {}
        out = zl.decode_attn(w.q.cuda(), k, v, btd, sl, page_size=16, scale=w.scale,
                             tree_mask=mask.cuda(), err_flags=err, **new)
        torch.cuda.synchronize()
        assert int(err.item()) == (zl.DEVERR_BAD_PAGE if fused else 0)
        got.append((out, k, v))
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    # a mapped page: nothing to report
    err = torch.zeros(1, dtype=torch.int32).cuda()
    zl.decode_attn(w.q.cuda(), w.k_pool.cuda(), w.v_pool.cuda(),
                   torch.from_numpy(w.block_table).cuda(), torch.from_numpy(w.seq_lens).cuda(),
                   page_size=16, scale=w.scale, tree_mask=mask.cuda(), err_flags=err,
                   k_new=kn.cuda(), v_new=vn.cuda())
    assert int(err.item()) == 0
    assert np.isfinite(out.float().cpu().numpy()).all()
