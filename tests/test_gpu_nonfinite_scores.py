"""Modified scores that are no finite numbers: the rows that see them are NaN,
however the call is cut and whichever kernel runs it, no page is called bad,
and every other row is within its bounds."""
import numpy as np
import pytest
import torch

import paged_decode_attention_gqa_gb300 as zl
from paged_decode_attention_gqa_gb300 import workloads as wl
from test_gpu_score_mods import random_trees, run, slopes_of

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# (8, 2, 1) to (32, 8, 2) are the 16-row kernel's, the others the tcgen05 kernel's with one
# row tile, (8, 2, 64) with two
SHAPES = [(8, 2, 1), (8, 2, 3), (32, 8, 2), (8, 2, 20), (64, 1, 1), (8, 2, 64)]


def case(Hq, Hkv, q_len, lens):
    return wl.random_case(3500 + q_len, B=len(lens), Hq=Hq, Hkv=Hkv, q_len=q_len, lens=lens,
                          poison=False)


def put(w, b, t, h, value, d=5):
    """K of cached token t (negative: from the end) of sequence b."""
    t += int(w.seq_lens[b]) if t < 0 else 0
    w.k_pool[w.block_table[b, t // 16], t % 16, h, d] = value


@pytest.mark.parametrize("ctas", [0, 1, 7, 60])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("Hq,Hkv,q_len", SHAPES)
def test_a_nonfinite_key(Hq, Hkv, q_len, value, ctas):
    """In the context, seen by every row of its kv head; and as one of the query
    tokens, seen by itself and what follows. (+inf times the query's component is
    +inf or -inf, a NaN row or a token of weight 0.)"""
    w = case(Hq, Hkv, q_len, [1500, 900, 700])
    w.q[..., 5] = w.q[..., 5].abs() + 0.5
    w.q[:, :, ::3, 5] *= -1                  # these heads' score is -inf
    put(w, 0, 400, 0, value)
    put(w, 1, -1 - q_len // 2, Hkv - 1, value)
    if value == INF:
        # the reference's own products with infinities lose its error bound: only where
        # it is NaN, and that the rest is finite
        out, lse = attend(w, num_ctas=ctas)
        sees = np.zeros((3, q_len, Hq), dtype=bool)
        g = Hq // Hkv
        sees[0, :, :g] = True
        sees[1, q_len - 1 - q_len // 2:, Hq - g:] = True
        sees[:, :, ::3] = False
        assert np.array_equal(torch.isnan(lse).cpu().numpy(), sees)
        assert np.array_equal(torch.isnan(out).all(3).cpu().numpy(), sees)
        assert np.array_equal(torch.isnan(out).any(3).cpu().numpy(), sees)
        return
    run(w, window=1600, num_ctas=ctas)
    run(w, slopes=slopes_of(Hq), num_ctas=ctas)


def attend(w, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros(w.B, w.q_len, w.Hq, device="cuda")
    kw = {**dict(alibi_slopes=torch.zeros(w.Hq, device="cuda")), **kw}
    out = zl.decode_attn(w.q.cuda(), w.k_pool.cuda(), w.v_pool.cuda(),
                         torch.from_numpy(w.block_table).cuda(),
                         torch.from_numpy(w.seq_lens).cuda(), page_size=16, scale=w.scale,
                         err_flags=err, lse=lse, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,q_len", SHAPES)
@pytest.mark.parametrize("max_seq_len", [0, 128])
def test_a_nan_query(Hq, Hkv, q_len, max_seq_len):
    w = case(Hq, Hkv, q_len, [128, 65, 100] if max_seq_len else [1500, 900, 700])
    w.q[1, q_len // 2, Hq - 1, 77] = NAN
    run(w, softcap=9.0, max_seq_len=max_seq_len)


@pytest.mark.parametrize("Hq,Hkv,q_len", SHAPES)
def test_a_nan_and_a_bad_page(Hq, Hkv, q_len):
    """A bad page still zeroes the rows that see it."""
    w = case(Hq, Hkv, q_len, [1500, 900, 700])
    for b in (0, 1):
        put(w, b, 300, 0, NAN)
    bt = w.block_table.copy()
    bt[0, 40] = w.num_pages
    run(w, block_table=bt, softcap=9.0, expect_bad=1)


@pytest.mark.parametrize("Hq,Hkv,q_len", SHAPES)
@pytest.mark.parametrize("ctas", [0, 7])
def test_infinite_scores_under_a_cap(Hq, Hkv, q_len, ctas):
    """The cap makes them finite: +-c, as for a very large score."""
    got = []
    for value in (INF, 1e36):
        w = case(Hq, Hkv, q_len, [1500, 900, 700])
        w.q[..., 5] = w.q[..., 5].abs() + 0.5
        w.q[:, :, ::3, 5] *= -1
        put(w, 0, 400, 0, value)
        got.append(attend(w, softcap=4.0, num_ctas=ctas))
    assert torch.isfinite(got[0][0]).all() and torch.isfinite(got[0][1]).all()
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("Hq,Hkv,q_len", SHAPES)
@pytest.mark.parametrize("ctas", [0, 7])
def test_rows_whose_scores_are_all_minus_infinity(Hq, Hkv, q_len, ctas):
    w = case(Hq, Hkv, q_len, [1500, 900, 700])
    w.k_pool[..., 5] = w.k_pool[..., 5].abs() + 0.5
    w.q[2, 0, 1, 5] = -INF
    out, lse = attend(w, num_ctas=ctas)
    assert torch.isneginf(lse[2, 0, 1]) and not out[2, 0, 1].any()
    lse[2, 0, 1] = 0
    assert torch.isfinite(lse).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, 1), (8, 2, 3), (32, 8, 2), (8, 2, 20)])
def test_weights_of_nan_rows(Hq, Hkv, q_len, window):
    """NaN for the tokens that a NaN row sees, and only for those."""
    w = case(Hq, Hkv, q_len, [1500, 90, 700])
    put(w, 0, -1 - q_len // 2, 0, NAN)
    mask = random_trees(np.random.default_rng(3), 3, q_len)
    old = torch.rand(3, Hkv, 1501, generator=torch.Generator().manual_seed(1))
    run(w, mask=mask, window=window, weights=old, softcap=9.0)
