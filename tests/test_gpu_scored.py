"""Decode with accumulated attention weights over 16- and 32-bit caches: the output is the
plain decode's bit for bit, the weights are within a bound that follows from the scores'
roundings."""
import numpy as np
import pytest
import torch

import compress_cases as cc
from gpu_cases import dev, pa_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


class Case:
    """A paged cache of random rows whose unused slots hold NaN."""

    def __init__(self, seed, lens, H, Hk, D, bs, dtype, gain=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.Hk, self.D, self.bs, self.dtype = np.asarray(lens, np.int32), H, Hk, D, bs, dtype
        self.bt, self.NB, _ = cc.tables(rng, lens, bs)
        self.scale = D ** -0.5
        d, dt = dev(), cc.TORCH[dtype]
        self.kc = torch.full((self.NB, bs, Hk, D), float("nan"), dtype=dt, device=d)
        self.vc = torch.full_like(self.kc, float("nan"))
        self.k, self.v = [], []
        for b, n in enumerate(self.lens):
            s = torch.from_numpy(cc.slots_of(self.bt[b], n, bs)).to(d)
            for cache, out in ((self.kc, self.k), (self.vc, self.v)):
                x = rng.standard_normal((n, Hk, D)).astype(np.float32)
                cache.view(-1, Hk, D)[s] = torch.from_numpy(x).to(d).to(dt)
                out.append(cc.stored(x, dtype))
        self.qv = rng.standard_normal((len(lens), H, D)).astype(np.float32) * np.float32(gain)
        self.q = torch.from_numpy(self.qv).to(d).to(dt)
        self.btd, self.lensd = torch.from_numpy(self.bt).to(d), torch.from_numpy(self.lens).to(d)

    def run(self, pa, mass, **kw):
        out = torch.full_like(self.q, float("nan"))
        pa.paged_attention_decode_scored(out, self.q, mass, self.kc, self.vc, self.btd, self.lensd, self.scale, **kw)
        return out

    def plain(self, pa, **kw):
        out = torch.full_like(self.q, float("nan"))
        pa.paged_attention_decode(out, self.q, self.kc, self.vc, self.btd, self.lensd, self.scale, **kw)
        return out

    def check(self, mass, before):
        """Scores are sums of D products: each is off by at most D 2^-23 of the absolute values
        summed, the weights by twice the largest such error of their row (themselves and the
        sum), exp2 and the sums of partitions add a few 2^-22; a weight below float32's least
        normal number, 2^-126, may be flushed to zero, and so may each of the up to 16 added up."""
        qs = cc.stored(self.qv, self.dtype)
        m = mass.double().cpu().numpy()
        for b, n in enumerate(self.lens):
            _, w, big, _ = cc.attention(qs[b], self.k[b], self.v[b], self.scale)
            rel = np.expm1(2 * big.max(1, initial=0.0) * (self.D + 1) * 2.0 ** -23)[:, None] + 8 * 2.0 ** -22
            want = before[b][:, :n] + cc.group_mass(w, self.Hk)
            tol = cc.group_mass(w * rel, self.Hk) + 2.0 ** -23 * want + 16 * 2.0 ** -126
            err = np.abs(m[b][:, :n] - want)
            assert (err <= tol).all(), (b, n, float((err - tol).max()))
            assert np.array_equal(m[b][:, n:], before[b][:, n:])


RAGGED = [1, 7, 0, 31, 33, 127, 128, 129, 300, 513, 1000, 1025]


@pytest.mark.parametrize("dtype,H,Hk,D,bs", [
    ("bf16", 8, 8, 128, 16), ("bf16", 32, 8, 128, 16), ("f16", 16, 2, 128, 8), ("bf16", 12, 1, 128, 128),
    ("f16", 6, 2, 64, 16), ("bf16", 32, 2, 128, 32), ("f32", 4, 4, 64, 4), ("f32", 8, 1, 128, 16), ("f32", 6, 2, 64, 1),
    ("f16", 5, 5, 128, 256)])
def test_scored_ragged(pa, dtype, H, Hk, D, bs):
    case = Case(100 + H + D + bs, RAGGED, H, Hk, D, bs, dtype)
    before = np.random.default_rng(9).random((len(RAGGED), Hk, 1040)).astype(np.float32)
    before[:4] = 0.0
    mass = torch.from_numpy(before).to(dev())
    out = case.run(pa, mass, max_context_len=1025)
    case.check(mass, before.astype(np.float64))
    assert torch.equal(out, case.plain(pa, max_context_len=1025))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("part", [128, 512])
def test_scored_partitions_and_peaks(pa, dtype, part):
    case = Case(5, [2000, 1, 128, 700, 0, 5000], 16, 2, 128, 16, dtype, gain=5.0)
    before = np.zeros((6, 2, 5000))
    mass = torch.zeros((6, 2, 5000), device=dev())
    out = case.run(pa, mass, partition_size=part)
    case.check(mass, before)
    assert torch.equal(out, case.plain(pa, partition_size=part))


def test_scored_weights_of_a_row_sum_to_its_group(pa):
    case = Case(6, [4096, 900], 32, 8, 128, 16, "bf16")
    mass = torch.zeros((2, 8, 4096), device=dev())
    for _ in range(3):
        case.run(pa, mass)
    # three passes of four heads a group; n sums of relative error 2^-20 each at most
    assert torch.allclose(mass.double().sum(-1).cpu(), torch.full((2, 8), 12.0, dtype=torch.float64), rtol=2e-5)


def test_scored_many_sequences(pa):
    lens = np.random.default_rng(8).integers(0, 50, 1200)
    case = Case(7, lens, 4, 2, 128, 16, "bf16")
    mass = torch.zeros((1200, 2, 50), device=dev())
    out = case.run(pa, mass, max_context_len=50)
    case.check(mass, np.zeros((1200, 2, 50)))
    assert torch.equal(out, case.plain(pa, max_context_len=50))


def test_scored_errors(pa):
    case = Case(10, [100, 60], 8, 2, 128, 16, "bf16")
    mass = torch.zeros((2, 2, 64), device=dev())
    case.run(pa, mass)
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT       # 100 tokens, mass holds 64: cut
    case.lens = np.array([64, 60], np.int32)
    case.k[0], case.v[0] = case.k[0][:64], case.v[0][:64]
    case.check(mass, np.zeros((2, 2, 64)))
    need = pa.decode_scored_workspace_bytes(2, 8, 2, 128, case.bt.shape[1] * 16, 0)
    with pytest.raises(pa.PagedAttnError) as e:
        case.run(pa, mass, workspace=torch.empty(need - 16, dtype=torch.uint8, device=dev()))
    assert e.value.status == pa.PA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        case.run(pa, mass[:1])
    with pytest.raises(TypeError):
        case.run(pa, mass.double())
