"""Plain forms of the operators around the 4-bit cache, in 64 bits (test
infrastructure; numpy, no code of the package)."""
import numpy as np
import torch

D, ROW = 128, 144
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
CODES = np.concatenate([MAGNITUDES, -MAGNITUDES])
# the numbers a scale byte stands for; 248 and above are an infinity and NaNs
_b = np.arange(256)
SCALES = np.where(_b < 8, (_b & 7) * 2.0 ** -17, (8 + (_b & 7)) * 2.0 ** ((_b >> 3) - 18.0))
SCALES[248:] = np.nan
TOP = int(np.flatnonzero(SCALES == 10240.0)[0])


def bf16(x):
    """float64 of a bf16 (or other) tensor."""
    return x.detach().double().cpu().numpy()


def quantise(x):
    """[..., 128] in 64 bits -> (codes [..., 128], scale bytes [..., 8])."""
    x = x.reshape(*x.shape[:-1], 8, 16)
    a = np.abs(x)
    bad = ~np.isfinite(x).all(-1)
    top = np.where(bad, 0, np.nan_to_num(a, posinf=0).max(-1))
    # nearest of the table's 6-folds (exact numbers in 64 bits), ties to the even byte
    six = 6 * SCALES[:TOP + 1]
    up = np.searchsorted(six, top).clip(max=TOP)
    down = (up - 1).clip(min=0)
    du, dd = np.abs(six[up] - top), np.abs(top - six[down])
    byte = np.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, down)
    s = SCALES[byte][..., None]
    a = np.minimum(np.where(bad[..., None], 0, a), 8 * s)  # (beyond 6 all the same)
    gaps = np.abs(a[..., None] - MAGNITUDES * s[..., None])
    order = [0, 2, 4, 6, 1, 3, 5, 7]  # the first of equal gaps: the even code
    code = np.array(order)[gaps[..., order].argmin(-1)]
    code = np.where(s == 0, 0, code) + 8 * np.signbit(x)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255, byte)
    return code.reshape(*code.shape[:-2], D), byte


def pack(k, v):
    """K and V [..., 128] in 64 bits -> rows [..., 144] uint8."""
    (ck, sk), (cv, sv) = quantise(k), quantise(v)
    parts = [c[..., 0::2] | (c[..., 1::2] << 4) for c in (ck, cv)] + [sk, sv]
    return np.concatenate(parts, -1).astype(np.uint8)


def unpack(rows):
    """rows [..., 144] uint8 -> K, V [..., 128] in 64 bits."""
    out = []
    for at, sc in ((0, 128), (64, 136)):
        b = rows[..., at:at + 64]
        code = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], D)
        x = CODES[code].reshape(*b.shape[:-1], 8, 16) * SCALES[rows[..., sc:sc + 8]][..., None]
        out.append(x.reshape(*b.shape[:-1], D))
    return out


def random_rows(g, *shape, spread=1.0):
    """bf16 K or V rows [..., 128], some blocks far larger or smaller than others."""
    x = g.standard_normal((*shape, 8, 16)) * np.exp(spread * g.standard_normal((*shape, 8, 1)))
    return torch.from_numpy(x.reshape(*shape, D)).to(torch.bfloat16)


class Cache:
    """A paged 4-bit cache on the CPU: pool [pages, P, Hkv, 144] (NHD) or HND, a shuffled
    block table, lengths."""

    def __init__(self, seed, lens, Hkv, P=16, layout="NHD", spare=3, fill=True, spread=1.0):
        self.g = g = np.random.default_rng(seed)
        self.lens, self.Hkv, self.P, self.layout = list(lens), Hkv, P, layout
        B = len(self.lens)
        need = [(L + P - 1) // P for L in self.lens]
        self.pages = sum(need) + spare
        perm = g.permutation(self.pages)
        self.bt = np.full((B, max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        shape = (self.pages, P, Hkv) if layout == "NHD" else (self.pages, Hkv, P)
        # bytes that no token wrote may be anything
        self.pool = g.integers(0, 256, (*shape, ROW), dtype=np.uint8)
        if fill:
            for b, L in enumerate(self.lens):
                if L:
                    k = bf16(random_rows(g, L, Hkv, spread=spread))
                    v = bf16(random_rows(g, L, Hkv, spread=spread))
                    self.put(b, np.arange(L), pack(k, v))

    def place(self, b, t):
        return self.bt[b, np.asarray(t) // self.P], np.asarray(t) % self.P

    def put(self, b, t, rows):
        page, slot = self.place(b, t)
        x = self.pool if self.layout == "NHD" else self.pool.transpose(0, 2, 1, 3)
        x[page, slot] = rows

    def rows(self, b, t, pool=None):
        page, slot = self.place(b, t)
        pool = self.pool if pool is None else pool
        x = pool if self.layout == "NHD" else pool.transpose(0, 2, 1, 3)
        return x[page, slot]

    def kv(self, b, pool=None):
        return unpack(self.rows(b, np.arange(self.lens[b]), pool))

    def on_gpu(self):
        return (torch.from_numpy(self.pool).cuda(), torch.from_numpy(self.bt).cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))


def attention(q, caches_kv, lens, scale):
    """q [B, q_len, Hq, 128] in 64 bits, per sequence (K, V) [L, Hkv, 128]. Returns out,
    lse and the bounds that decode_attn_q4's may be off by (see tolerance)."""
    B, n, Hq, _ = q.shape
    out, lse = np.zeros_like(q), np.full((B, n, Hq), -np.inf)
    t_out, t_lse = np.zeros_like(q), np.zeros((B, n, Hq))
    for b in range(B):
        k, v = caches_kv[b]
        g = Hq // k.shape[1]
        for i in range(n):
            see = lens[b] - n + 1 + i
            if see <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[:see, h // g], v[:see, h // g]
                x = kk @ q[b, i, h] * scale
                m = x.max()
                p = np.exp(x - m)
                lse[b, i, h] = m + np.log(p.sum())
                p /= p.sum()
                out[b, i, h] = p @ vv
                size = (np.abs(kk) @ np.abs(q[b, i, h])).max() * scale
                t_out[b, i, h], t_lse[b, i, h] = tolerance(out[b, i, h], p @ np.abs(vv), size,
                                                           np.abs(x).max(), see,
                                                           np.abs(vv).max())
    return out, lse, t_out, t_lse


def tolerance(out, weighted, size, score, L, top):
    """How far the kernel's row may be off, from its roundings.

    A score: products of fp16 numbers, exact, summed in fp32 over 8 instructions of 16
    (at most 16 roundings or truncations, 2^-23 each, of the sum of magnitudes ``size``),
    two products and one sum of about its own size (2^-23 each of score + 16, the base's
    distance). That is e; a weight is off by e and the normaliser's e, relatively, and by
    2^-21 for the exponentials. P is rounded to fp16 (2^-11, or an absolute 2^-25 where
    the largest P is at least 2^7: 2^-32 of it for each of L tokens), sums and merges in
    32 bits (2^-20), the output to bf16 (2^-8)."""
    e = 16 * 2.0 ** -23 * size + 3 * 2.0 ** -23 * (score + 16)
    rel = 2.0 ** -11 + 2.0 ** -20 + 2.0 ** -21 + 2 * e
    t = 2.0 ** -8 * np.abs(out) + (1 + 2.0 ** -8) * (rel * weighted + L * 2.0 ** -32 * top)
    return t, e + 2.0 ** -20 + 2.0 ** -22 * score


def norm_rope(x, weight, eps, pos, freq, axis_of, interleaved, scale=1.0):
    """x [B, n, H, 128] in 64 bits; pos [axes, B, n]; freq radians per position."""
    x = x.copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    n = len(freq)
    if n == 0:
        return x
    angle = np.stack([pos[a].astype(np.longdouble) * np.longdouble(f)
                      for a, f in zip(axis_of, freq)], -1)
    co, si = (np.cos(angle).astype(np.float64)[:, :, None] * scale,
              np.sin(angle).astype(np.float64)[:, :, None] * scale)
    one, two = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved
                else (slice(0, n), slice(n, 2 * n)))
    a, b = x[..., one].copy(), x[..., two].copy()
    x[..., one], x[..., two] = a * co - b * si, b * co + a * si
    return x


def norm_rope_tolerance(want, size):
    """bf16's rounding (2^-8), and 32-bit roundings before it: the sum of squares (128
    terms, 2^-20 at most), root, three products, two of them in a difference (2^-22), and
    sines and cosines of an angle that 32 bits hold to 2^-25 of a half-turn, pi times it
    (2^-23), with 2^-22 of their own: 2^-19 of the pair's size in all."""
    return 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * 2.0 ** -19 * size
