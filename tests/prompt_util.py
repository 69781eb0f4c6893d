"""Plain fp64 forms of the attention layers' prompt side, and what its outputs may be off by."""
import math

import numpy as np
import torch

import kv_util as ku


def attend(q, k, v, window, sm_scale, x=None):
    """One request: rows q, k, v (fp64 [n, h, d]) behind earlier positions x (fp64 [2, h, L, d] or None)."""
    if x is None:
        x = np.zeros((2, k.shape[1], 0, k.shape[2]))
    return ku.attend_request(x, q, k, v, window, sm_scale)


# Error budget of an output:
#   the final rounding to bf16      2^-8 |o|
#   the weights p, to bf16          2^-8 A      (A = sum p |v|), and fp32 sums and exponentials 2^-18 A
#   the scores                      ds = (d + 8) 2^-22 max sum |q k| sm_scale (fp32 products and sums in any
#                                   order, a factor 4 for the tensor cores' own), which moves o by 2 ds A
# and of the log-sum-exp: ds + 2^-20 (1 + |lse|).
def bounds(o, lse, a, worst, d):
    ds = (d + 8) * 2.0 ** -22 * worst
    ob = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -18 + 2 * ds[..., None]) * a + 1e-30
    lb = ds + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return ob, lb


def rows_of(total, h_q, h_kv, d, seed, k_scale=1.0, pad=0):
    """Rows of a fused projection (bf16 tensor on the CPU) and views of its fp64 values as q, k, v."""
    g = np.random.RandomState(seed + 77)
    x = g.standard_normal((total, (h_q + 2 * h_kv) * d + pad))
    x[:, h_q * d:(h_q + h_kv) * d] *= k_scale
    t, f = ku.bf16(x)
    return t, split(f, h_q, h_kv, d)


def split(z, h_q, h_kv, d):
    cut = lambda a, h: z[:, a:a + h * d].reshape(z.shape[0], h, d) if isinstance(z, np.ndarray) \
        else z[:, a:a + h * d].unflatten(1, (h, d))
    return cut(0, h_q), cut(h_q * d, h_kv), cut((h_q + h_kv) * d, h_kv)


def cu_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def scale_of(d):
    return float(np.float32(1.0 / math.sqrt(d)))


def dev32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)
