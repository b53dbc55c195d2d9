"""Rotary positions of negative frequencies on the GPU: the mirror image of positive ones, as exact far out."""
import numpy as np
import pytest
import torch

import step_cases as sc
from gpu_cases import dev, pa_mod
from test_gpu_rotary import assert_close, projection

pytestmark = pytest.mark.gpu

POS = np.array([0, 1, 77, 4097, 131071, (1 << 24) + 1, 1234567891, (1 << 31) - 1, -1, -70000, -(1 << 31)], np.int32)


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def frequencies(rng):
    """Magnitudes from above a turn a position down to 1e-12, and nothing."""
    f = 10.0 ** rng.uniform(-12, 1.3, 64)
    f[:5] = 1e-4, 3e-6, 2e-9, 2 * np.pi, 0.0
    return f


def rotate(pa, x, pos, f):
    out = torch.empty_like(x)
    pa.rotary_embedding(out, None, x, None, torch.from_numpy(pos).to(dev()), torch.from_numpy(f).to(dev()))
    return out


def test_negative_frequencies_against_the_formula(pa):
    rng = np.random.default_rng(3)
    x, vals = projection(rng, len(POS), 6, 128, "f32")
    f = -frequencies(rng)
    assert_close(rotate(pa, x, POS, f), vals, POS, f, 1.0, False, "f32")
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_negative_frequencies_mirror_positions(pa, dtype):
    """A frequency of the other sign at a position of the other sign is the same angle, bit for bit."""
    rng = np.random.default_rng(4)
    pos = POS[:-1]
    x, _ = projection(rng, len(pos), 3, 128, dtype)
    f = frequencies(rng)
    f[1::2] *= -1
    assert torch.equal(rotate(pa, x, pos, -f), rotate(pa, x, -pos, f))
    assert pa.get_device_error() == 0
