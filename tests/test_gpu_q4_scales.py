"""Attention over a 4-bit cache that others wrote: every scale byte that stands for a number,
those above what kv_append_q4 writes among them, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from plain_q4 import ROW, SCALES, Cache, bf16, pack, random_rows
from test_gpu_q4_attn import check, queries, run

pytestmark = pytest.mark.gpu
WAYS = [dict(), dict(num_ctas=3), dict(max_seq_len=700)]


def cache(seed, k_scales, v_scales, lens=(700, 33, 100), Hkv=2, P=16):
    """Random codes, scale bytes drawn from the two lists; a code 6 in every block."""
    c = Cache(seed, lens, Hkv, P, fill=False)
    for b, L in enumerate(lens):
        rows = c.g.integers(0, 256, (L, Hkv, ROW), dtype=np.uint8)
        rows[..., 0:128:8] = 0x7F  # codes 6 and -6
        rows[..., 128:136] = c.g.choice(k_scales, (L, Hkv, 8))
        rows[..., 136:] = c.g.choice(v_scales, (L, Hkv, 8))
        c.put(b, np.arange(L), rows)
    return c


ORDINARY = list(range(100, 124))  # 2^-5 .. 1.9
LARGE = list(range(0xE0, 0xF8))   # 8192 .. 61440: times 6 beyond fp16 from 0xE3 on
SMALL = list(range(0, 24))        # 0 .. 2^-12


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("q_len,Hq", [(1, 8), (3, 8), (6, 6)])
def test_values_beyond_fp16(q_len, Hq, way):
    c = cache(50 + q_len, ORDINARY, LARGE)
    check(c, queries(c, q_len, Hq, 0.5), **way)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("q_len,Hq", [(1, 8), (3, 8), (6, 6)])
def test_keys_beyond_fp16(q_len, Hq, way):
    """Queries as small as the keys are large: scores of a few units."""
    c = cache(60 + q_len, LARGE, ORDINARY)
    check(c, queries(c, q_len, Hq, 2.0 ** -18), **way)


@pytest.mark.parametrize("way", WAYS)
def test_the_smallest_values(way):
    """Steps of 2^-18, the format's least: exact in the products as well."""
    c = cache(70, SMALL, SMALL)
    check(c, queries(c, 2, 8, 2.0 ** 12), **way)


def test_every_scale_of_one_value():
    """A token for each of the 248 scales, V all one code: with equal scores the output is the
    mean of the values; the last query token alone sees them all."""
    c = Cache(71, [248], 1, fill=False)
    rows = np.zeros((248, 1, ROW), np.uint8)
    rows[..., 64:128] = 0x77
    rows[..., 136:] = np.arange(248, dtype=np.uint8)[:, None, None]
    c.put(0, np.arange(248), rows)
    out, lse, err = run(c, queries(c, 248 - 120, 2))
    assert err == 0
    for i in range(128):
        mean = 6 * SCALES[:121 + i].mean()
        # bf16's half step; P is the same power of two for each token: sums of up to 248
        # numbers in 32 bits, and rcp (2^-23), lie within 2^-15
        assert (np.abs(out[0, i] - mean) <= mean * (2.0 ** -8 + 2.0 ** -14)).all()
        assert np.abs(lse[0, i] - np.log(121 + i)).max() <= 2.0 ** -18


def test_what_the_package_writes_is_as_it_was():
    """The largest numbers that kv_append_q4 writes beside ordinary ones."""
    c = Cache(72, [300, 20], 2, fill=False)
    for b, L in enumerate(c.lens):
        k = bf16(random_rows(c.g, L, 2))
        v = bf16(random_rows(c.g, L, 2))
        v[::7, 0, :16] *= 1e30
        c.put(b, np.arange(L), pack(k, v))
    check(c, queries(c, 2, 8))
    assert torch.isfinite(torch.from_numpy(c.kv(0)[1])).all()
