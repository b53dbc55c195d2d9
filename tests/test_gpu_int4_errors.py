"""4-bit decode where its inputs are at their worst: bad block ids, whose tokens count with score and
value 0, and V scales far apart, within the bounds that the decode states."""
import numpy as np
import pytest
import torch

import compress_cases as cc
from gpu_cases import dev, pa_mod
from test_gpu_int4 import Case, bound, parts, score_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


@pytest.mark.parametrize("H,Hk,D,bs,bad", [(8, 2, 128, 16, (2, 5)), (12, 1, 64, 8, (0, 12)), (8, 2, 128, 128, (0,))])
def test_bad_blocks_read_as_zeros(pa, H, Hk, D, bs, bad):
    """Some blocks of one sequence, its last and partly filled one among them; then every one."""
    n = 100
    case = Case(np.random.default_rng(71), [n, 60], H, Hk, D, bs, "bf16")
    want = case.run(pa)[1].clone()
    for j, blocks in enumerate((bad, range(-(-n // bs)))):
        for i in blocks:
            b = case.bt[0, i]
            case.t["bt"][0, i] = (case.NB, -1, 1 << 30)[(i + j) % 3]
            case.kc[b], case.vc[b], case.par[b] = 0, 0, 0
            case.k[0][i * bs:(i + 1) * bs], case.v[0][i * bs:(i + 1) * bs] = 0.0, 0.0
        mass = torch.zeros((2, Hk, n), device=dev())
        out = case.run(pa, mass)
        assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
        case.check(out, mass)
        assert torch.equal(out[1], want)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5])
def test_one_v_row_far_larger_than_the_others(pa, size, D):
    """A V row at the format's end among small ones. Products of weights and V scales are within 2^-33 of
    the largest weight (at most 1 of the softmax's sum, which is 1 at least in the same units) times a power
    of two that is at most twice the largest V scale, on top of the bound of the other tests; a code is at
    most 15, and every token adds its error."""
    n = 300
    case = Case(np.random.default_rng(73), [n, n], 8, 2, D, 16, "f16", gain=2.0, v_size=size)
    for b, t in ((0, 17), (1, 250)):
        codes, s, z = cc.cache_rows(np.linspace(-6e4, 6e4, D).astype(np.float32))
        blk, off = case.bt[b, t // 16], t % 16
        for h in range(2):
            case.vc[blk, h, off], case.par[blk, h, off, 2], case.par[blk, h, off, 3] = codes, s, z
            case.v[b][t, h] = cc.values(codes, s, z)
            # its key opposes the queries, so its weight is small for most heads
            k = -8.0 * np.sign(case.q[b, 4 * h:4 * h + 4].sum(0))
            kc, ks, kz = cc.cache_rows(k.astype(np.float32))
            case.kc[blk, h, off], case.par[blk, h, off, 0], case.par[blk, h, off, 1] = kc, ks, kz
            case.k[b][t, h] = cc.values(kc, ks, kz)
    for k in ("kc", "vc", "par"):
        case.t[k] = torch.from_numpy(getattr(case, k)).to(dev())
    mass = torch.zeros((2, 2, n), device=dev())
    out = case.run(pa, mass).double().cpu().numpy()
    qs = cc.stored(case.q, "f16")
    for b in range(2):
        ref, w, _, _ = cc.attention(qs[b], case.k[b], case.v[b], case.scale)
        tol = bound(ref, score_error(qs[b], case, b), parts(case, b, w), "f16")
        tol = tol + (1 + cc.EPS["f16"]) * 15 * n * 2.0 ** -33 * 2 * float(s)
        err = np.abs(out[b] - ref)
        assert (err <= tol).all(), (b, float((err - tol).max()))
    # each head's weights sum to 1, off by float32 sums of n terms and by exp2
    assert np.abs(mass.double().cpu().numpy().sum(-1) - 4).max() <= 4 * (n * 2.0 ** -24 + 2.0 ** -20)


@pytest.mark.parametrize("B,n,Hk,D", [(18, 430, 3, 64), (18, 430, 3, 128), (1, 1900, 1, 128), (2, 1000, 1, 64)])
@pytest.mark.parametrize("width", [0, 5])
def test_weights_leave_the_output_as_it_is(pa, B, n, Hk, D, width):
    """Bit for bit, also where mass holds fewer tokens than the tables and max_context_len, so that the
    longest context the call may have differs with and without it: as many partials a row as one warp
    joins, or as four do, and more."""
    rng = np.random.default_rng(B + n)
    lens = rng.integers(n // 4, n, B)
    lens[0] = n
    case = Case(rng, lens, 8 * Hk, Hk, D, 16, "bf16", reserve=130)
    for max_ctx in (0, 4 * n, n):
        mass = torch.zeros((B, Hk, n + width), device=dev())
        out = case.run(pa, mass, max_context_len=max_ctx)
        assert torch.equal(out, case.run(pa, max_context_len=max_ctx))
        case.check(out, mass)
    assert pa.get_device_error() == 0
