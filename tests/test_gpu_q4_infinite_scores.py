"""Scores that leave 32 bits, over a 4-bit cache: above their range the row is NaN, below
it the token weighs nothing, however the call is cut."""
import numpy as np
import pytest
import torch

from plain_q4 import Cache, bf16, pack, random_rows
from test_gpu_q4_attn import run

pytestmark = pytest.mark.gpu
WAYS = [dict(), dict(num_ctas=1), dict(num_ctas=7), dict(max_seq_len=1500), dict(max_seq_len=64)]
LOUD = 61440.0  # the largest value a cached element takes when it is written


def cache(seed, lens, sign, P=16, Hkv=2):
    """Keys of zeros, but sign[b][t] * LOUD in element 5 (sign 0: zeros)."""
    c = Cache(seed, lens, Hkv, P, fill=False)
    vs = []
    for b, L in enumerate(lens):
        k = np.zeros((L, Hkv, 128))
        k[:, :, 5] = LOUD * np.asarray(sign[b])[:, None]
        v = bf16(random_rows(c.g, L, Hkv, spread=0.0))
        c.put(b, np.arange(L), pack(k, v))
        vs.append(c.kv(b)[1])
    return c, vs


def loud_queries(c, q_len, Hq):
    """Element 5 so large that LOUD times it leaves 32 bits, in every second head; ordinary
    in the others."""
    q = torch.zeros(len(c.lens), q_len, Hq, 128)
    q[..., 0::2, 5] = 3e38
    q[..., 1::2, 5] = 2.0 ** -20
    return q.to(torch.bfloat16)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("q_len,Hq", [(1, 4), (1, 16), (3, 4), (5, 6)])
def test_scores_below_32_bits_weigh_nothing(q_len, Hq, way):
    """Whole tiles of them at the start, in the middle, at the end; single ones; all."""
    rng = np.random.default_rng(5)
    lens = [1500, 700, 64, 333, 40]
    signs = [np.zeros(L) for L in lens]
    signs[0][:800] = -1
    signs[1][200:] = -1
    signs[1][-q_len:] = 0
    signs[2][:] = -rng.integers(0, 2, 64)
    signs[2][0] = 0
    signs[3][:] = -1                     # every token: a row that sees none
    signs[4][1:] = -1
    c, vs = cache(80, lens, signs)
    q = loud_queries(c, q_len, Hq)
    out, lse, err = run(c, q, **way)
    assert err == 0 and not np.isnan(out).any() and not np.isnan(lse).any()
    g = Hq // 2
    for b, L in enumerate(lens):
        for i in range(q_len):
            see = L - q_len + 1 + i
            for h in range(Hq):
                left = np.arange(see)
                x = np.zeros(see)
                if h % 2 == 0:
                    left = left[signs[b][:see] == 0]
                    x = x[:len(left)]
                else:
                    x = signs[b][:see] * LOUD * 2.0 ** -20 * 128 ** -0.5
                if len(left) == 0:
                    assert not out[b, i, h].any() and lse[b, i, h] == -np.inf
                    continue
                v = vs[b][left, h // g]
                p = np.exp(x)
                want, size = p @ v / p.sum(), p @ np.abs(v) / p.sum()
                # P rounded to fp16, sums in 32 bits, the output to bf16
                tol = 2.0 ** -8 * np.abs(want) + 1.01 * (2.0 ** -11 + 2.0 ** -18) * size
                assert (np.abs(out[b, i, h] - want) <= tol).all()
                assert abs(lse[b, i, h] - np.log(p.sum())) <= 2.0 ** -17


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("q_len,Hq", [(1, 4), (3, 4), (5, 6)])
def test_a_score_above_32_bits(q_len, Hq, way):
    """One token's; among scores below 32 bits as well. Rows before it keep their numbers."""
    lens = [1500, 700, 64]
    signs = [np.zeros(L) for L in lens]
    signs[0][801] = 1
    signs[1][:300] = -1
    signs[1][650] = 1
    signs[2][-1] = 1                     # seen by the last query token alone
    c, _ = cache(81, lens, signs)
    out, lse, err = run(c, loud_queries(c, q_len, Hq), **way)
    assert err == 0
    bad = np.zeros(lse.shape, bool)
    bad[:2, :, 0::2] = True
    bad[2, -1, 0::2] = True
    assert (np.isnan(lse) == bad).all() and (np.isnan(out).all(-1) == bad).all()
    assert np.isfinite(out[~bad]).all() and np.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("way", WAYS)
def test_the_least_numbers_of_32_bits(way):
    """Scores next to the border, on its near side: one row whose only scores lie there."""
    L = 300
    c, vs = cache(82, [L], [-np.ones(L)], Hkv=1)
    q = torch.zeros(1, 1, 2, 128)
    # times LOUD, 128^-1/2 and log2(e): 3.3e38 and 2e38
    q[0, 0, :, 5] = torch.tensor([3.3e38, 2e38]) / (LOUD * 128 ** -0.5 * 1.4427)
    q = q.to(torch.bfloat16)
    assert (bf16(q)[..., 5] * LOUD * 128 ** -0.5 * 1.4427 < 3.4e38).all()
    out, lse, err = run(c, q, **way)
    assert err == 0
    v = vs[0][:, 0]
    low, high = v.min(0), v.max(0)
    for h in range(2):
        x = -bf16(q)[0, 0, h, 5] * LOUD * 128 ** -0.5
        assert abs(lse[0, 0, h] - x) <= 2.0 ** -20 * abs(x)
        # All scores are equal. How many tokens a part holds is lost in its log-sum-exp (a
        # step of 32 bits is 2^103 at 2e38, the log of 300 tokens 8.2), so parts weigh the same
        # whatever they hold: a mean of the tokens, but not one with equal weights.
        y = out[0, 0, h]
        assert y.any() and (y >= low - 2.0 ** -8 * np.abs(low)).all()
        assert (y <= high + 2.0 ** -8 * np.abs(high)).all()
