"""Plain 64-bit forms of the cache-compression operators, for their tests: numpy on the
host, written from the formulas and sharing no code with the library."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = {k: float(torch.finfo(t).eps) for k, t in TORCH.items()}


def stored(x, dtype):
    """float64 values of x after rounding to dtype (nearest, ties to even)."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TORCH[dtype]).double().numpy()


# ---- the 4-bit format -------------------------------------------------------------

def quantise(x):
    """Rows x [..., D] (float32-exact values): codes uint8 [..., D], scale and zero float16 [...]."""
    x = np.asarray(x, np.float32)
    nan = np.isnan(x).any(-1)
    c = np.clip(np.nan_to_num(x, nan=0.0, posinf=65504.0, neginf=-65504.0), np.float32(-65504.0), np.float32(65504.0))
    lo, hi = c.min(-1), c.max(-1)
    zero = lo.astype(np.float16)
    scale = ((hi - lo).astype(np.float32) / np.float32(15.0)).astype(np.float16)
    s, z = scale.astype(np.float32)[..., None], zero.astype(np.float32)[..., None]
    with np.errstate(all="ignore"):
        n = np.rint(((c - z).astype(np.float32) / np.where(s > 0, s, np.float32(1.0))).astype(np.float32))
    n = np.where(s > 0, np.clip(n, 0.0, 15.0), 0.0)
    n = np.where(nan[..., None], 0.0, n)
    scale, zero = (np.where(nan, np.float16(np.nan), a).astype(np.float16) for a in (scale, zero))
    return n.astype(np.uint8), scale, zero


def pack(n):
    return n[..., 0::2] | (n[..., 1::2] << 4)


def unpack(b):
    out = np.empty((*b.shape[:-1], 2 * b.shape[-1]), np.uint8)
    out[..., 0::2] = b & 15
    out[..., 1::2] = b >> 4
    return out


def cache_rows(x):
    """Rows x [..., D] as (packed codes [..., D / 2], scale, zero)."""
    n, s, z = quantise(x)
    return pack(n), s, z


def values(codes, scale, zero):
    """float64 values of packed codes [..., D / 2] with scale and zero [...]."""
    return (unpack(codes).astype(np.float64) * scale.astype(np.float64)[..., None]
            + zero.astype(np.float64)[..., None])


# ---- attention ----------------------------------------------------------------------

def attention(q, k, v, scale):
    """One sequence, float64: q [H, D], k and v [n, Hk, D] -> (out [H, D], weights [H, n],
    absolute values of the products of each score summed [H, n], weighted |v| [H, D])."""
    H, D = q.shape
    n, Hk, _ = k.shape
    if n == 0:
        return np.zeros((H, D)), np.zeros((H, 0)), np.zeros((H, 0)), np.zeros((H, D))
    G = H // Hk
    kh, vh = np.repeat(k, G, 1), np.repeat(v, G, 1)
    x = np.einsum("hd,nhd->hn", q, kh) * scale
    e = np.exp(x - x.max(1, keepdims=True))
    w = e / e.sum(1, keepdims=True)
    big = np.einsum("hd,nhd->hn", np.abs(q), np.abs(kh)) * abs(scale)
    return np.einsum("hn,nhd->hd", w, vh), w, big, np.einsum("hn,nhd->hd", w, np.abs(vh))


def group_mass(w, Hk):
    """Weights [H, n] summed over the query heads of each kv head: [Hk, n]."""
    H, n = w.shape
    return w.reshape(Hk, H // Hk, n).sum(1)


# ---- eviction -----------------------------------------------------------------------

def evict(mass, c, keep, recent):
    """Indices that stay of one (sequence, kv head): mass [>= c]."""
    n = min(c, keep)
    r = min(recent, n)
    m = mass[:c - r].astype(np.float64)
    m = np.where(np.isnan(m), -np.inf, m)
    nan = np.isnan(mass[:c - r])
    order = np.lexsort((np.arange(c - r), nan, -m))       # heaviest first; NaN after -inf; ties to the lower index
    return np.concatenate([np.sort(order[:n - r]), np.arange(c - r, c)]).astype(np.int64)


# ---- paged storage --------------------------------------------------------------------

def tables(rng, lens, bs, spare=3, reserve=0):
    """Shuffled block tables of `lens` tokens a sequence (+ reserve blocks each), padded with
    -1, and the number of blocks."""
    need = [-(-int(n) // bs) + reserve for n in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb).astype(np.int32)
    width = max(max(need), 1)
    bt = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[at:at + k]
        at += k
    return bt, nb, perm[at:]


def slots_of(bt_row, n, bs):
    t = np.arange(n)
    return bt_row[t // bs].astype(np.int64) * bs + t % bs
