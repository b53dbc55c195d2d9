"""Rotary positions on the GPU, alone and with the scatter, against the 64-bit formula."""
import numpy as np
import pytest
import torch

import compress_cases as cc
import step_cases as sc
from gpu_cases import dev, pa_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def projection(rng, T, heads, D, dtype):
    """A fused projection's output on the device, and its values."""
    x = rng.standard_normal((T, heads, D)).astype(np.float32) * 3
    return torch.from_numpy(x).to(dev()).to(cc.TORCH[dtype]), cc.stored(x, dtype)


def assert_close(got, x, pos, f, factor, inter, dtype):
    ref = sc.rotate(x, pos, f, factor, inter)
    tol = sc.rotate_bound(x, ref, pos, f, factor, inter, cc.EPS[dtype])
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err - tol).max())


SHAPES = [(1, 1, 1, 64, 64), (64, 32, 8, 128, 128), (37, 6, 2, 128, 32), (300, 3, 3, 64, 48), (19, 5, 1, 80, 80),
          (7, 2, 1, 1024, 1008), (5, 4, 4, 16, 16), (2500, 4, 1, 128, 64)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,Hk,D,rd", SHAPES)
def test_rotary_embedding(pa, dtype, inter, T, H, Hk, D, rd):
    """Views of a projection; out of place, into other views, and in place."""
    rng = np.random.default_rng(T + D)
    x, vals = projection(rng, T, H + 2 * Hk, D, dtype)
    q, k = x[:, :H], x[:, H:H + Hk]
    pos = rng.integers(0, 100000, T).astype(np.int32)
    pos[0] = 0 if T > 1 else 5
    f = pa.rotary_frequencies(rd, 1e4)
    pt, ft = torch.from_numpy(pos).to(dev()), torch.from_numpy(f).to(dev())
    qo, ko = torch.full((T, H, D), 9.0, dtype=x.dtype, device=dev()), torch.full((T, Hk, D), 9.0, dtype=x.dtype, device=dev())
    pa.rotary_embedding(qo, ko, q, k, pt, ft, 1.25, inter)
    assert_close(qo, vals[:, :H], pos, f, 1.25, inter, dtype)
    assert_close(ko, vals[:, H:H + Hk], pos, f, 1.25, inter, dtype)
    wide = torch.full((T, H + Hk + 2, D), 7.0, dtype=x.dtype, device=dev())
    pa.rotary_embedding(wide[:, 1:H + 1], wide[:, H + 1:H + 1 + Hk], q, k, pt, ft, 1.25, inter)
    assert torch.equal(wide[:, 1:H + 1], qo) and torch.equal(wide[:, H + 1:H + 1 + Hk], ko)
    assert (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()
    v = x[:, H + Hk:].clone()
    pa.rotary_embedding(q, k, q, k, pt, ft, 1.25, inter)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(x[:, H + Hk:], v)
    only = torch.empty_like(qo)
    pa.rotary_embedding(only, None, q, None, pt, ft, interleaved=inter)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,Hk,D,rd,bs", [(1, 1, 1, 64, 64, 1), (64, 32, 8, 128, 128, 16), (37, 6, 2, 128, 32, 12),
                                            (300, 3, 3, 64, 48, 256), (1100, 8, 8, 128, 64, 16)])
def test_write_rotary(pa, dtype, inter, T, H, Hk, D, rd, bs):
    """Caches as paged_kv_write leaves them with the rotated keys, bit for bit; padding and slots out of range."""
    rng = np.random.default_rng(T + D + bs)
    x, _ = projection(rng, T, H + 2 * Hk, D, dtype)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    NB = -(-T // bs) + 2
    slots = rng.choice(NB * bs, T, replace=False).astype(np.int32)
    if T > 8:
        slots[[3, T - 1]], slots[5] = -1, NB * bs
    st = torch.from_numpy(slots).to(dev())
    pt = torch.from_numpy(rng.integers(0, 9000, T).astype(np.int32)).to(dev())
    ft = torch.from_numpy(pa.rotary_frequencies(rd)).to(dev())
    qo, ko = torch.empty((T, H, D), dtype=x.dtype, device=dev()), torch.empty((T, Hk, D), dtype=x.dtype, device=dev())
    pa.rotary_embedding(qo, ko, q, k, pt, ft, interleaved=inter)
    want = [torch.full((NB, bs, Hk, D), 3.0, dtype=x.dtype, device=dev()) for _ in range(2)]
    if (Hk * D * x.element_size()) % 16 == 0:
        pa.paged_kv_write(ko, v.contiguous(), st, *want)
    got, q2 = [torch.full_like(w, 3.0) for w in want], torch.empty_like(qo)
    pa.get_device_error()
    pa.paged_kv_write_rotary(q2, q, k, v, pt, ft, st, *got, interleaved=inter)
    assert torch.equal(q2, qo) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert pa.get_device_error() == (pa.PA_DEVERR_SLOT if T > 8 else 0)


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "by_turns", "by_index"])
def test_far_positions(pa, scaling):
    """Positions to the end of 32 bits and negative ones, where a float32 angle has lost its turns; frequencies
    above a turn a position and of nothing."""
    f = pa.rotary_frequencies(128, 5e5, scaling, 8.0 if scaling else 1.0)
    f[5], f[6], f[7] = 0.0, 17.3, -2.0
    pos = np.array([0, 1, 4097, 131071, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -1, -70000, -(1 << 31)], np.int32)
    rng = np.random.default_rng(1)
    x, vals = projection(rng, len(pos), 4, 128, "f32")
    out = torch.empty_like(x)
    pa.rotary_embedding(out, None, x, None, torch.from_numpy(pos).to(dev()), torch.from_numpy(f).to(dev()))
    assert_close(out, vals, pos, f, 1.0, False, "f32")


def test_python_refusals(pa):
    x = torch.zeros((4, 6, 128), device=dev(), dtype=torch.bfloat16)
    q, k, v = x[:, :2], x[:, 2:4], x[:, 4:]
    pos, f = torch.zeros(4, dtype=torch.int32, device=dev()), torch.zeros(64, dtype=torch.float64, device=dev())
    out, cache = torch.zeros((4, 2, 128), device=dev(), dtype=torch.bfloat16), torch.zeros((2, 16, 2, 128), device=dev(), dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int32, device=dev())
    ok = (out, q, k, v, pos, f, slots, cache, cache)
    for i, bad, exc in ((0, out[:3], ValueError), (0, out.float(), TypeError), (1, q.transpose(1, 2), ValueError),
                        (2, k[:, :1], ValueError), (4, pos.long(), TypeError), (4, pos[:3], ValueError), (5, f.float(), TypeError),
                        (5, f[None], ValueError), (6, slots[:2], ValueError), (7, cache[..., :64].contiguous(), ValueError),
                        (8, cache.half(), TypeError), (3, v[:, :, ::2], ValueError)):
        args = list(ok)
        args[i] = bad
        with pytest.raises(exc):
            pa.paged_kv_write_rotary(*args)
    with pytest.raises(ValueError, match="both"):
        pa.rotary_embedding(out, None, q, k, pos, f)
    with pytest.raises(pa.PagedAttnError):                # rotary_dim 24
        pa.rotary_embedding(out, None, q, None, pos, f[:12])
    assert pa.get_device_error() == 0
