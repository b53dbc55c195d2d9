"""Plain forms of the operators of a serving step (block tables and slot maps, rotary
positions, the block-scaled 8-bit cache), for their tests: numpy on the host, written from the
formulas and sharing no code with the library."""
from __future__ import annotations

import numpy as np

# ---- the E4M3 format ------------------------------------------------------------------


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


E4M3 = _e4m3_table()
_POS = E4M3[:127]                                     # 0 .. 448, ascending
_MID = (_POS[1:] + _POS[:-1]) / 2


def encode(x):
    """E4M3 codes of float64 x: nearest, ties to the even code, +-448 beyond, NaN to 0x7F (either sign)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    i = np.searchsorted(_MID, np.nan_to_num(a), side="left")
    tie = (i < len(_MID)) & (np.nan_to_num(a) == _MID[np.minimum(i, len(_MID) - 1)])
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    code = i + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def same_codes(a, b):
    """Equal, NaN codes of either sign counting as one."""
    nan = (a & 127) == 127
    return np.array_equal(nan, (b & 127) == 127) and np.array_equal(a[~nan], b[~nan])


def scale_for(amax):
    """The smallest 2^e, e >= -100, with amax <= 448 * 2^e."""
    e = -100
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def write_blocks(kc, vc, sc, k, v, slots):
    """paged_kv_write_fp8_block on numpy arrays, in place: codes [NB, Hk, bs, D], scales float32
    [NB, Hk, 2], k and v float64 [T, Hk, D]."""
    NB, Hk, bs, _ = kc.shape
    blocks = {}
    for t, s in enumerate(slots):
        if 0 <= s < NB * bs:
            blocks.setdefault(int(s) // bs, []).append((t, int(s) % bs))
    for b, tokens in blocks.items():
        at, off = [t for t, _ in tokens], [o for _, o in tokens]
        for j, (x, c) in enumerate(((k, kc), (v, vc))):
            for h in range(Hk):
                new = x[at, h]
                a = np.abs(new[np.isfinite(new)])
                s = scale_for(a.max(initial=0.0))
                old = float(sc[b, h, j])
                if 0 not in off and 0 < old <= 2.0 ** 126:
                    while s < old:
                        s *= 2
                    if s > old:                       # the product in float32: scales may be foreign ones
                        with np.errstate(all="ignore"):
                            x32 = E4M3[c[b, h]].astype(np.float32) * np.float32(old / s)
                        c[b, h] = encode(x32)
                c[b, h, off] = encode(new / s)
                sc[b, h, j] = s


def block_values(c, sc, j):
    """float64 values [NB, Hk, bs, D] of codes with the scales of K (j = 0) or V (j = 1)."""
    return E4M3[c] * sc[:, :, j].astype(np.float64)[:, :, None, None]


# ---- rotary positions -------------------------------------------------------------------

def rotate(x, positions, inv_freq, factor=1.0, interleaved=False):
    """float64 x [T, heads, D] with its first 2 * len(inv_freq) channels turned."""
    half = len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * inv_freq
    c, s = (factor * f(a)[:, None] for f in (np.cos, np.sin))
    y = np.array(x, np.float64)
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def rotate_bound(x, y, positions, inv_freq, factor, interleaved, eps):
    """How far a rotated channel may be off: cosine and sine by 2^-23 (their float32 rounding, the
    function's, the reduced angle's) and the angle's 64-bit rounding, each product and the factor by a
    float32 rounding, and one rounding to the type; untouched channels by nothing."""
    half = len(inv_freq)
    a = np.abs(np.asarray(positions, np.float64)[:, None] * inv_freq)[:, None]
    rel = abs(factor) * (2.0 ** -23 + a * 2.0 ** -50 + 3 * 2.0 ** -24)
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    tol = np.zeros_like(y)
    tol[..., one] = tol[..., two] = (np.abs(x[..., one]) + np.abs(x[..., two])) * rel
    live = np.zeros(x.shape[-1], bool)
    live[:2 * half] = True
    # an f16 below 2^-14 is a multiple of 2^-24; for the other types the last term is nothing
    return np.where(live, tol + (np.abs(y) + tol) * eps / 2 + eps * 2.0 ** -15, 0.0)


# ---- block tables and slot maps -----------------------------------------------------------

def append(table, lens, new, free, num_free, T, bs, NB):
    """paged_blocks_append request by request: (table, new lens, num_free, start, slots, positions, error
    kinds), with copies of what changes."""
    table, lens, err = table.copy(), lens.copy(), set()
    B, MB = table.shape
    height = num_free if 0 <= num_free <= len(free) else 0
    if height != num_free:
        err.add("free")
    left, dry, rows = height, False, 0
    start, slots, pos = np.zeros(B + 1, np.int32), np.full(T, -1, np.int32), np.zeros(T, np.int32)
    for b in range(B):
        c, n = int(lens[b]), int(new[b])
        first, rows = rows, rows + max(n, 0)
        start[b + 1] = min(rows, T)
        if c < 0 or n < 0 or c + n > MB * bs or (n > 0 and rows > T):
            err.add("context")
            continue
        held = -(-c // bs)
        need = -(-(c + n) // bs) - held
        if need > 0 and (dry or need > left):
            dry = True
            err.add("free")
            continue
        for j in range(need):
            left -= 1
            e = int(free[left])
            if not 0 <= e < NB:
                err.add("block")
                e = -1
            table[b, held + j] = e
        for i in range(n):
            e = int(table[b, (c + i) // bs])
            if not 0 <= e < NB:
                err.add("block")
            else:
                slots[first + i] = e * bs + (c + i) % bs
            pos[first + i] = c + i
        lens[b] = c + n
    return table, lens, left, start, slots, pos, err


def release(table, lens, finished, free, num_free, bs, NB):
    """paged_blocks_release request by request: (new lens, free, num_free, error kinds)."""
    lens, free, err, full = lens.copy(), free.copy(), set(), False
    B, MB = table.shape
    top = num_free if 0 <= num_free <= len(free) else 0
    if top != num_free:
        err.add("free")
    for b in range(B):
        if not finished[b]:
            continue
        c = int(lens[b])
        if not 0 <= c <= MB * bs:
            err.add("context")
            continue
        n = -(-c // bs)
        if n and (full or top + n > len(free)):
            full = True
            err.add("free")
            continue
        for j in range(n):
            e = int(table[b, j])
            if not 0 <= e < NB:
                err.add("block")
                e = -1
            free[top] = e
            top += 1
        lens[b] = 0
    return lens, free, top, err
