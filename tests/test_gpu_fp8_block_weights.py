"""What the block-scaled decode's weights lose before they meet V: no more than float32 does, whatever the
type of the outputs."""
import numpy as np
import pytest
import torch

import compress_cases as cc
from gpu_cases import dev, pa_mod
from test_gpu_fp8_block import RUNS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def bound(q, k, v, scale, dtype):
    """(output, bound) of one sequence whose query has one channel that is not zero, so a score is one exact product
    of an f16 and a code, times two factors: off by 2^-22 of itself and, less the reference, of the largest. A term of
    an output's sum is off by its weight's error -- its own score's and the sum's, e^(2 dx) --, by 2^-20 (exp2, the
    weights as two f16, 22 bits) and by 2^-22 for each of n + 8 additions (the tensor cores', the sum's, the
    joins'); below 2^-22 of the largest weight times the largest V scale it is within 2^-33 of that. One rounding to
    the type, an f16's to multiples of 2^-24 at least."""
    n = k.shape[0]
    ref, _, big, wv = cc.attention(q, k, v, scale)
    dx = 2 * big.max(1, initial=0.0)[:, None] * 2.0 ** -22
    rel = np.expm1(2 * dx) + 2.0 ** -20 + (n + 8) * 2.0 ** -22
    eps, small = cc.EPS[dtype], n * 2.0 ** -33 * 448 * 2 * max(2 * np.abs(v).max(initial=0.0) / 448, 2.0 ** -100)
    return ref, np.abs(ref) * eps / 2 + (1 + eps) * (rel * wv + small) + eps * 2.0 ** -14


@pytest.mark.parametrize("limit", [0, RUNS])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hk,D,bs", [(8, 2, 128, 16), (12, 4, 64, 8), (16, 1, 128, 16), (12, 1, 64, 32)])
def test_weights_keep_float32s_precision(pa, dtype, H, Hk, D, bs, limit):
    """Few tokens of V of either sign: where they cancel, an output is far smaller than its terms, and its own
    rounding hides nothing of theirs."""
    rng = np.random.default_rng(71 + H + D)
    case = Case(rng, [2, 3, 4, 5, 7, 9, 17, 40] * 4, H, Hk, D, bs, dtype)
    case.scale = 1.0
    case.q[:, :, np.arange(D) != 5] = 0
    case.t["q"] = torch.from_numpy(case.q).to(dev()).to(cc.TORCH[dtype])
    got, q = case.run(pa, max_context_len=limit).double().cpu().numpy(), cc.stored(case.q, dtype)
    off = []
    for b in range(len(case.lens)):
        ref, tol = bound(q[b], *case.kv(b), case.scale, dtype)
        off.append(np.abs(got[b] - ref) - tol)
    assert max(x.max() for x in off) <= 0, (max(x.max() for x in off), sum((x > 0).sum() for x in off))
    assert pa.get_device_error() == 0
