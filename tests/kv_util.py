"""Plain fp64 forms of the paged 8-bit cache's operators, and seeded caches to run them on."""
import math

import numpy as np
import torch


def _values():
    c = np.arange(256)
    ex, man = (c >> 3) & 15, c & 7
    mag = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    mag[(c & 127) == 127] = np.nan
    return np.where(c & 128, -mag, mag)


VALUES = _values()                       # the value of each e4m3 code
_POS = VALUES[:127]                      # 0 .. 448, increasing with the code


def encode(x):
    """fp64 -> e4m3 codes: nearest, ties to the even code, +-448 beyond, NaN to a NaN code."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - _POS[lo], _POS[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(mag == 0, 0, code) | (np.signbit(x) * 128)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def scale_for(amax):
    """2^ceil(log2(amax / 448)), at least 2^-100 (fp64 arrays, by comparison with powers of two)."""
    amax = np.asarray(amax, np.float64)
    _, e = np.frexp(amax)
    s = np.ldexp(1.0, e - 9)
    s = np.where(amax > 448.0 * s, 2 * s, s)
    return np.where(amax > 0, np.maximum(s, 2.0 ** -100), 2.0 ** -100)


class Cache:
    """A seeded cache of `layers` layers on the CPU, requests' pages shuffled over the pool."""

    def __init__(self, lens, h_q, h_kv, d, page_tokens, layers=1, room=None, seed=0, fill="normal", spare=2):
        g = np.random.RandomState(seed)
        room = lens if room is None else room
        T = page_tokens
        need = [-(-n // T) for n in room]
        self.h_q, self.h_kv, self.d, self.T, self.lens = h_q, h_kv, d, T, list(lens)
        self.pages = sum(need) + spare
        perm = g.permutation(self.pages)
        self.table = np.full((len(lens), max(1, max(need, default=1))), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = perm[at:at + n]
            at += n
        x = g.standard_normal((self.pages, layers, 2, h_kv, T, d))
        x *= np.exp2(g.randint(-3, 4, (self.pages, layers, 2, h_kv, 1, 1)))
        s = scale_for(np.abs(x).max((-2, -1)))                       # [pages, layers, 2, h_kv]
        self.kv = encode(x / s[..., None, None])
        self.scale = np.ascontiguousarray(s.swapaxes(2, 3)).astype(np.float32)
        if fill == "garbage":            # what lies past a request's end: NaN codes and wild scales
            used = np.zeros(self.pages, bool)
            for r, n in enumerate(lens):
                for j in range(-(-n // T)):
                    p = self.table[r, j]
                    used[p] = True
                    self.kv[p, :, :, :, max(0, n - j * T):] = 127 + 128 * (j % 2)
            self.kv[~used] = 127
            self.scale[~used] = np.inf

    def dense(self, r, layer, length=None):
        """fp64 [2, h_kv, length, d] of request r."""
        n = self.lens[r] if length is None else length
        ids = self.table[r, :-(-n // self.T)]
        x = VALUES[self.kv[ids, layer]] * self.scale[ids, layer].astype(np.float64).swapaxes(1, 2)[..., None, None]
        return x.transpose(1, 2, 0, 3, 4).reshape(2, self.h_kv, -1, self.d)[:, :, :n]


def attend_request(x, q, k, v, window, sm_scale):
    """x [2, h, L, d]; q [n, h_q, d]; k, v [n, h, d] or None (fp64).  -> o, lse, and the sizes that error
    bounds are made of: A = sum p |v| and the largest sum |q k| sm_scale over what a row sees."""
    n, h_q, d = q.shape
    h, L = x.shape[1:3]
    g = h_q // h
    kk = np.concatenate([x[0], k.transpose(1, 0, 2)], 1) if k is not None else x[0]
    vv = np.concatenate([x[1], v.transpose(1, 0, 2)], 1) if k is not None else x[1]
    qq = q.reshape(n, h, g, d)
    s = np.einsum("nhgd,htd->nhgt", qq, kk) * sm_scale
    mag = np.einsum("nhgd,htd->nhgt", np.abs(qq), np.abs(kk)) * abs(sm_scale)
    t = np.arange(kk.shape[1])[None]
    at = (L + np.arange(n))[:, None] if k is not None else np.full((n, 1), L - 1)
    see = t <= at
    if window:
        see &= t > at - window
    see = np.broadcast_to(see[:, None, None, :], s.shape)
    s = np.where(see, s, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    top = np.where(np.isinf(top), 0.0, top)
    p = np.where(see, np.exp(s - top), 0.0)
    total = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[..., 0]
    p = p / np.where(total > 0, total, 1.0)
    vv = np.where(see.any((0, 1, 2))[None, :, None], vv, 0.0)        # what no row sees is not there
    o = np.einsum("nhgt,htd->nhgd", p, vv)
    a = np.einsum("nhgt,htd->nhgd", p, np.abs(vv))
    worst = np.where(see, mag, 0.0).max(-1, initial=0.0)
    return (o.reshape(n, h_q, d), lse.reshape(n, h_q), a.reshape(n, h_q, d), worst.reshape(n, h_q))


# Error budget of an output (u = 2^-8 is bf16's unit roundoff):
#   the final rounding              u |o|
#   the weights p, to 12 bits       2^-12 A     (A = sum p |v|), and fp32 sums and exponentials 2^-18 A
#   the scores                      ds = (d + 8) 2^-22 max sum |q k| sm_scale (fp32 products and sums in any
#                                   order, a factor 4 for the tensor cores' own), which moves o by 2 ds A
# and of the log-sum-exp: ds + 2^-20 (1 + |lse|).
def attend_bounds(o, lse, a, worst, d):
    ds = (d + 8) * 2.0 ** -22 * worst
    ob = 2.0 ** -8 * np.abs(o) + (2.0 ** -12 + 2.0 ** -18 + 2 * ds[..., None]) * a + 1e-30
    lb = ds + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return ob, lb


def append_request(cache, r, layer, k, v):
    """Commits rows (fp64 [n, h, d]) to request r of a Cache, by the definition, page by page."""
    L, T = cache.lens[r], cache.T
    x = np.stack([k, v]).transpose(0, 2, 1, 3)                       # [2, h, n, d]
    at, n = 0, x.shape[2]
    while at < n:
        j, t0 = divmod(L + at, T)
        m = min(T - t0, n - at)
        p = cache.table[r, j]
        part = x[:, :, at:at + m]
        mag = np.where(np.isfinite(part), np.abs(part), 0.0)
        was = cache.scale[p, layer].astype(np.float64).T if t0 else np.zeros((2, cache.h_kv))
        now = np.maximum(was, scale_for(mag.max((-2, -1))))
        if t0:
            old = VALUES[cache.kv[p, layer, :, :, :t0]] * (was / now)[..., None, None]
            grew = (now > was)[..., None, None]
            cache.kv[p, layer, :, :, :t0] = np.where(grew, encode(old), cache.kv[p, layer, :, :, :t0])
        cache.kv[p, layer, :, :, t0:t0 + m] = encode(part / now[..., None, None])
        cache.scale[p, layer] = now.T
        at += m


def bf16(x):
    """fp array -> (bf16 tensor, the fp64 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


def gpu_cache(cache, dev, window=0, sm_scale=None):
    from speculative_decoding_hybrid_gb300.kvcache import Kv8Cache
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    return Kv8Cache(torch.from_numpy(cache.kv).to(dev), torch.from_numpy(cache.scale).to(dev), cache.h_q, status,
                    window=window, sm_scale=sm_scale)


def default_scale(d):
    return float(np.float32(1.0 / math.sqrt(d)))
