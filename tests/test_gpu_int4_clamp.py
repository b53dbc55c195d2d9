"""The clamp of the 4-bit scatter to +-65504, bit for bit: rows so narrow that the code of a
channel past the clamp depends on it."""
import numpy as np
import pytest
import torch

import compress_cases as cc
from gpu_cases import dev, pa_mod
from test_gpu_int4 import assert_cache, write_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def narrow_rows(rng, T, Hk, D):
    """Rows of a narrow range next to 65504, or next to -65504, some of whose channels lie beyond."""
    low = rng.choice(np.array([65340.0, 65460.0, 65472.0, 65488.0, 65490.0, 65503.0], np.float32), (T, Hk, 1))
    x = low + rng.random((T, Hk, D), dtype=np.float32) * rng.choice(np.array([5.0, 13.0, 20.0], np.float32), (T, Hk, 1))
    past = rng.choice(np.array([65504.0, 65505.0, 65519.0, 65520.0, 70000.0, 3e38, np.inf], np.float32), (T, Hk, D))
    x = np.where(rng.random((T, Hk, D)) < 0.1, past, x)
    return (x * np.where(rng.random((T, Hk, 1)) < 0.3, -1.0, 1.0)).astype(np.float32)


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hk,D,bs", [(40, 3, 128, 16), (40, 1, 64, 8), (1500, 3, 128, 32), (2100, 2, 64, 16)])
def test_channels_past_the_clamp(pa, src, T, Hk, D, bs):
    """Few rows (8 channels a lane) and many (32)."""
    rng = np.random.default_rng(T + D)
    NB = -(-T // bs)
    slots = rng.permutation(NB * bs)[:T].astype(np.int32)
    got, want = write_case(pa, narrow_rows(rng, T, Hk, D), narrow_rows(rng, T, Hk, D), slots, NB, bs, src)
    assert_cache(got, want)
    assert pa.get_device_error() == 0


def test_a_channel_past_the_clamp_reads_as_the_clamp(pa):
    """65460 and 65480 with one 70000: zero 65472, scale f16(44 / 15), and code round(32 / scale) = 11 for
    65504; 65490 to 65503 with an infinity: zero 65504, so every code is 0."""
    a = np.full((1, 1, 64), 65460.0, np.float32)
    a[0, 0, 20:40], a[0, 0, 50] = 65480.0, 70000.0
    b = np.linspace(65490.0, 65503.0, 64).astype(np.float32).reshape(1, 1, 64)
    b[0, 0, 3] = np.inf
    (kc, vc, par), _ = write_case(pa, a, b, np.zeros(1, np.int32), 1, 8, "f32")
    assert cc.unpack(kc.cpu().numpy())[0, 0, 0, 50] == 11 and not vc[0, 0, 0].any()
    out = [torch.empty((1, 1, 64), device=dev()) for _ in range(2)]
    pa.paged_kv_read_int4(*out, torch.zeros(1, dtype=torch.int32, device=dev()), kc, vc, par)
    scale = float(np.float16(44.0 / 15.0))
    assert float(out[0][0, 0, 50]) == np.float32(11.0 * scale + 65472.0) and bool((out[1] == 65504.0).all())
