"""Plain 64-bit forms of the modified-score attention, the cache eviction and
the path commit, written from their formulas, with the error each 32-bit step
of the kernels may add (for tolerances that follow from arithmetic alone)."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

E32 = 2.0 ** -24   # half a step of fp32, relative
EB = 2.0 ** -8     # half a step of bf16, relative


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def mask_bits(mask, q_len) -> np.ndarray:
    """int32 words [B, q, W] -> bool [B, q, q]."""
    w = np.asarray(mask.cpu()).view(np.uint32)
    bits = (w[..., None] >> np.arange(32, dtype=np.uint32)) & 1
    return bits.reshape(w.shape[0], w.shape[1], -1)[:, :, :q_len].astype(bool)


@dataclass
class Attention:
    out: np.ndarray        # [B, q, Hq, D]
    lse: np.ndarray        # [B, q, Hq]
    weights: np.ndarray    # [B, Hkv, T] sums of the softmax weights
    out_tol: np.ndarray    # allowed error of each element
    lse_tol: np.ndarray
    weights_tol: np.ndarray
    bad: int               # device error bits


def attention(q, k, v, block_table, seq_lens, *, scale, softcap=0.0, slopes=None, window=0,
              mask=None, tokens=None, num_pages=None, decay=None, old=None) -> Attention:
    """q [B, q, Hq, D]; k, v pools [pages, P, Hkv, D] (NHD), float64 numpy.
    tokens: length of the weights rows (None: no weights, no limit from them)."""
    B, q_len, Hq, D = q.shape
    pages, P, Hkv, _ = k.shape
    num_pages = pages if num_pages is None else num_pages
    g = Hq // Hkv
    cap = block_table.shape[1] * P
    if tokens is not None:
        cap = min(cap, tokens)
    T = tokens or 1
    out = np.zeros((B, q_len, Hq, D))
    lse = np.full((B, q_len, Hq), -np.inf)
    wts = np.zeros((B, Hkv, T))
    out_tol, lse_tol, w_tol = np.zeros_like(out), np.zeros_like(lse), np.zeros_like(wts)
    bits = None if mask is None else mask_bits(mask, q_len)
    err = 0
    for b in range(B):
        L = int(seq_lens[b])
        if L < 0 or L > cap:
            err |= 2
            continue
        if L == 0:
            continue
        ctx = L - q_len
        t = np.arange(L)
        pos_t = t.copy()
        for i in range(q_len):
            if bits is not None:
                depth = np.maximum(bits[b].sum(1) - 1, 0)
                pos = ctx + depth[i]
                j = t - ctx
                d = j >= 0
                pos_t = np.where(d, ctx + depth[np.clip(j, 0, q_len - 1)], t)
                vis = np.where(d, bits[b, i, np.clip(j, 0, q_len - 1)], t <= pos)
            else:
                pos = ctx + i
                vis = t <= pos
            dist = pos - pos_t
            if window:
                vis = vis & (dist < window)
            tv = np.flatnonzero(vis)
            if tv.size == 0:
                continue
            pg = block_table[b, tv // P]
            if ((pg < 0) | (pg >= num_pages)).any():
                err |= 1
                continue  # zeros, -inf, no weights
            for kh in range(Hkv):
                kk, vv = k[pg, tv % P, kh], v[pg, tv % P, kh]
                for h in range(kh * g, (kh + 1) * g):
                    dots = kk @ q[b, i, h]
                    mag = (np.abs(kk) @ np.abs(q[b, i, h])) * scale
                    s = dots * scale
                    # 128 products summed in fp32, one scaling
                    ds = (D + 4) * E32 * mag
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                        # cap_tanh: a few roundings of values up to 1, times the cap
                        ds = ds + softcap * 2.0 ** -21
                    bias = 0.0
                    if slopes is not None:
                        bias = slopes[h] * dist[tv]
                        s = s - bias
                    # fma and base subtraction round values of this size; ex2 2^-22
                    ds = ds + (np.abs(s) + np.abs(bias) + np.abs(s).max()) * 4 * E32 + 2.0 ** -21
                    m = s.max()
                    e = np.exp(s - m)
                    den = e.sum()
                    p = e / den
                    dp = p * 1.01 * (ds + (p * ds).sum() + (L / 16 + 64) * E32)
                    # P is rounded to bf16 for the tensor core (EB), then V is summed in
                    # fp32 and the result rounded to bf16
                    absv = np.abs(vv)
                    out[b, i, h] = p @ vv
                    out_tol[b, i, h] = (EB * np.abs(out[b, i, h]) + (1 + EB) * (
                        EB * (p @ absv) + dp @ absv + (L / 16 + 200) * E32 * (p @ absv)) + 1e-30)
                    lse[b, i, h] = m + np.log(den)
                    lse_tol[b, i, h] = ((p * ds).sum() + (L / 16 + 64) * E32
                                        + 8 * E32 * (abs(lse[b, i, h]) + abs(m)))
                    if tokens is not None:
                        wts[b, kh, tv] += p
                        w_tol[b, kh, tv] += dp + 4 * E32 * p
        if tokens is not None and old is not None:
            base = decay * old[b, :, :L] if decay else 0.0
            wts[b, :, :L] += base
            w_tol[b, :, :L] += (q_len * g + 2) * E32 * np.abs(wts[b, :, :L])
    if tokens is not None and old is not None:  # at and past the end, and bad lengths: as it was
        for b in range(B):
            L = int(seq_lens[b])
            L = L if 0 <= L <= cap else 0
            wts[b, :, L:] = old[b, :, L:]
            w_tol[b, :, L:] = 0
    return Attention(out, lse, wts, out_tol, lse_tol, w_tol, err)


def check(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - ref) <= tol))
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {at}: "
                             f"{got[at]!r}, expected {ref[at]!r} +- {tol[at]:.3g}")


def evict(k, v, weights, block_table, seq_lens, *, page_size, budget, sink, recent, num_pages,
          dst_table=None, weights_out=None):
    """Copies of the pools (NHD, any dtype; v may be None) and of the weights
    after the eviction, the kept lists, the new lengths and the error bits."""
    P = page_size
    k, v = k.copy(), None if v is None else v.copy()
    src_k, src_v = k.copy(), None if v is None else v.copy()
    w_in = weights
    w_out = (weights if weights_out is None else weights_out).copy()
    B, Hkv, T = weights.shape
    kept = np.full((B, Hkv, budget), -1, dtype=np.int32)
    new = np.array(seq_lens, dtype=np.int32).copy()
    dst = block_table if dst_table is None else dst_table
    err = 0
    for b in range(B):
        L = int(seq_lens[b])
        if L < 0 or L > block_table.shape[1] * P or L > T or min(L, budget) > dst.shape[1] * P:
            err |= 2
            continue
        new[b] = min(L, budget)
        for h in range(Hkv):
            keep = list(range(L))
            if L > budget:
                mid = range(sink, L - recent)
                key = {t: (-np.inf if np.isnan(w_in[b, h, t]) else w_in[b, h, t]) for t in mid}
                isnan = {t: bool(np.isnan(w_in[b, h, t])) for t in mid}
                order = sorted(mid, key=lambda t: (isnan[t], -key[t], t))
                keep = sorted(list(range(sink)) + order[:budget - sink - recent]
                              + list(range(L - recent, L)))
            kept[b, h, :len(keep)] = keep
            w_out[b, h, :len(keep)] = w_in[b, h, keep]
            for j, t in enumerate(keep):
                if dst_table is None and j == t:
                    continue
                ps, pd = block_table[b, t // P], dst[b, j // P]
                if not (0 <= ps < num_pages and 0 <= pd < num_pages):
                    err |= 1
                    continue
                k[pd, j % P, h] = src_k[ps, t % P, h]
                if v is not None:
                    v[pd, j % P, h] = src_v[ps, t % P, h]
    return k, v, w_out, kept, new, err


def commit(k, v, block_table, seq_lens, path, accepted, *, page_size, q_len, num_pages):
    P = page_size
    k, v = k.copy(), None if v is None else v.copy()
    src_k, src_v = k.copy(), None if v is None else v.copy()
    new = np.array(seq_lens, dtype=np.int32).copy()
    err = 0
    for b in range(len(new)):
        L, n = int(seq_lens[b]), int(accepted[b])
        ok = True
        if L < q_len or L > block_table.shape[1] * P:
            err |= 2
            ok = False
        if n < 0 or n > min(q_len, path.shape[1]) or any(
                not 0 <= x < q_len for x in path[b, :max(n, 0)]):
            err |= 16
            ok = False
        if not ok:
            continue
        ctx = L - q_len
        new[b] = ctx + n
        for j in range(n):
            ts, td = ctx + int(path[b, j]), ctx + j
            if ts == td:
                continue
            ps, pd = block_table[b, ts // P], block_table[b, td // P]
            if not (0 <= ps < num_pages and 0 <= pd < num_pages):
                err |= 1
                continue
            k[pd, td % P] = src_k[ps, ts % P]
            if v is not None:
                v[pd, td % P] = src_v[ps, ts % P]
    return k, v, new, err
