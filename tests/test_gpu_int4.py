"""The 4-bit cache on the GPU against plain 64-bit forms: scatter and read-back bit for
bit, decode within a bound that follows from its roundings (see bound())."""
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


def rows(rng, shape, kind="plain"):
    x = rng.standard_normal(shape).astype(np.float32) * (0.5 + rng.random(shape[-1])).astype(np.float32)
    if kind == "k":
        x += rng.standard_normal(shape[-1]).astype(np.float32)
    return x.astype(np.float32)


# ---------------------------------------------------------------------------- write, read

def write_case(pa, x_k, x_v, slots, NB, bs, src):
    T, Hk, D = x_k.shape
    d = dev()
    kc = torch.full((NB, Hk, bs, D // 2), 0xA5, dtype=torch.uint8, device=d)
    vc = torch.full_like(kc, 0x5A)
    par = torch.full((NB, Hk, bs, 4), 7.0, dtype=torch.float16, device=d)
    pa.paged_kv_write_int4(torch.from_numpy(x_k).to(d).to(cc.TORCH[src]), torch.from_numpy(x_v).to(d).to(cc.TORCH[src]),
                           torch.as_tensor(slots, device=d), kc, vc, par)
    torch.cuda.synchronize()
    ek, ev = np.full((NB, Hk, bs, D // 2), 0xA5, np.uint8), np.full((NB, Hk, bs, D // 2), 0x5A, np.uint8)
    ep = np.full((NB, Hk, bs, 4), 7.0, np.float16)
    sk, sv = cc.stored(x_k, src).astype(np.float32), cc.stored(x_v, src).astype(np.float32)
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= NB * bs:
            continue
        b, o = slot // bs, slot % bs
        ek[b, :, o], ep[b, :, o, 0], ep[b, :, o, 1] = cc.cache_rows(sk[t])
        ev[b, :, o], ep[b, :, o, 2], ep[b, :, o, 3] = cc.cache_rows(sv[t])
    return (kc, vc, par), (ek, ev, ep)


def assert_cache(got, want):
    for g, w in zip(got[:2], want[:2]):
        assert np.array_equal(g.cpu().numpy(), w)
    g, w = got[2].cpu().numpy(), want[2]
    assert np.array_equal(np.isnan(g), np.isnan(w))
    assert np.array_equal(g[~np.isnan(w)], w[~np.isnan(w)])


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hk,D,bs", [(1, 1, 128, 16), (37, 8, 128, 16), (19, 3, 64, 8), (130, 5, 64, 256)])
def test_write_is_bit_exact(pa, src, T, Hk, D, bs):
    rng = np.random.default_rng(7 + T + D)
    NB = -(-T // bs) + 2
    slots = rng.choice(NB * bs, T, replace=False).astype(np.int32)
    if T > 4:
        slots[[1, T // 2]] = -1
    got, want = write_case(pa, rows(rng, (T, Hk, D), "k"), rows(rng, (T, Hk, D)), slots, NB, bs, src)
    assert_cache(got, want)
    assert pa.get_device_error() == 0


def test_write_special_rows(pa):
    """Constant rows, rows of +-0, tiny, huge, infinite and NaN elements, exact ties between codes."""
    D = 128
    base = np.linspace(-3.0, 4.5, D).astype(np.float32)
    r = [np.zeros(D), np.full(D, -0.0), np.full(D, 2.7), base * 1e-9, base * 1e-5, base * 1e30, base * 2e4,
         np.where(np.arange(D) == 5, np.inf, base), np.where(np.arange(D) == 9, -np.inf, base),
         np.where(np.arange(D) == 77, np.nan, base), np.full(D, np.nan), np.full(D, np.inf),
         np.arange(D) % 31 * 0.5, np.where(np.arange(D) == 0, 7.5, 0.25 * (np.arange(D) % 30))]
    x = np.stack(r).astype(np.float32)[:, None, :]
    got, want = write_case(pa, x, x[::-1].copy(), np.arange(len(r), dtype=np.int32), 1, 16, "f32")
    assert_cache(got, want)
    # what is read back: the formula's values, NaN rows whole
    out_k = torch.full((len(r), 1, D), 123.0, device=dev())
    out_v = torch.full_like(out_k, 123.0)
    pa.paged_kv_read_int4(out_k, out_v, torch.arange(len(r), dtype=torch.int32, device=dev()), *got)
    for out, codes, i in ((out_k, want[0], 0), (out_v, want[1], 2)):
        ref = cc.values(codes[0, :, :len(r)], want[2][0, :, :len(r), i], want[2][0, :, :len(r), i + 1])
        assert np.array_equal(out.cpu().numpy()[:, 0], ref[0].astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dst", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hk,D,bs", [(1, 1, 128, 16), (53, 8, 128, 32), (21, 3, 64, 8)])
def test_read_back(pa, dst, T, Hk, D, bs):
    """Repeated slots, -1 and out-of-range ones; rows of those stay as they were."""
    rng = np.random.default_rng(70 + T)
    d = dev()
    NB = 4
    kc = rng.integers(0, 256, (NB, Hk, bs, D // 2), dtype=np.uint8)
    vc = rng.integers(0, 256, (NB, Hk, bs, D // 2), dtype=np.uint8)
    par = rng.standard_normal((NB, Hk, bs, 4)).astype(np.float16)
    slots = rng.integers(0, NB * bs, T).astype(np.int32)
    if T > 8:
        slots[3], slots[5], slots[7] = -1, NB * bs, -9
    ko = torch.full((T, Hk, D), 5.0, dtype=cc.TORCH[dst], device=d)
    vo = torch.full_like(ko, 6.0)
    pa.paged_kv_read_int4(ko, vo, torch.as_tensor(slots, device=d), torch.from_numpy(kc).to(d),
                          torch.from_numpy(vc).to(d), torch.from_numpy(par).to(d))
    assert pa.get_device_error() == (pa.PA_DEVERR_SLOT if T > 8 else 0)
    for out, codes, i, stay in ((ko, kc, 0, 5.0), (vo, vc, 2, 6.0)):
        ref = np.full((T, Hk, D), stay, np.float32)
        for t, s in enumerate(slots):
            if 0 <= s < NB * bs:
                ref[t] = cc.values(codes[s // bs, :, s % bs], par[s // bs, :, s % bs, i],
                                   par[s // bs, :, s % bs, i + 1]).astype(np.float32)
        assert torch.equal(out.cpu(), torch.from_numpy(ref).to(cc.TORCH[dst]))


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 8), (128, 32)])
def test_write_and_read_many_rows(pa, src, D, bs):
    """Enough rows for the wide form of both kernels: ties between codes, constant rows, infinities and
    NaN among them, slots of -1 and out of range, a last CTA that is not full."""
    rng = np.random.default_rng(D)
    T, Hk, d = 5501, 3, dev()
    x = np.stack([rows(rng, (T, Hk, D), "k"), rows(rng, (T, Hk, D))])
    x[:, 10:400] = rng.integers(-8, 24, (2, 390, Hk, D)) * np.float32(0.5)     # ties, halves of a step
    x[:, 10:400, :, 0], x[:, 10:400, :, 1] = 0.0, 7.5
    x[0, 500], x[1, 501], x[0, 502, 1, 7], x[1, 503, 2, 5], x[0, 504, 0, 9] = 1.25, 0.0, np.nan, np.inf, -np.inf
    x[:, 600:700] *= np.float32(1e-6)
    x[:, 700:800] *= np.float32(1e4)
    NB = -(-T // bs) + 1
    slots = rng.choice(NB * bs, T, replace=False).astype(np.int32)
    slots[[0, 77, T - 1]] = -1, NB * bs, -5
    kc = torch.full((NB, Hk, bs, D // 2), 0xA5, dtype=torch.uint8, device=d)
    vc, par = torch.full_like(kc, 0x5A), torch.full((NB, Hk, bs, 4), 7.0, dtype=torch.float16, device=d)
    src_t = [torch.from_numpy(a).to(d).to(cc.TORCH[src]) for a in x]
    pa.paged_kv_write_int4(*src_t, torch.from_numpy(slots).to(d), kc, vc, par)
    want = [t.cpu().numpy() for t in (torch.full_like(kc, 0xA5), torch.full_like(vc, 0x5A), torch.full_like(par, 7.0))]
    live = np.flatnonzero((slots >= 0) & (slots < NB * bs))
    b, o = slots[live] // bs, slots[live] % bs
    back = []
    for i, a in enumerate(x):
        codes, sc, ze = cc.cache_rows(cc.stored(a[live], src).astype(np.float32))
        want[i][b, :, o] = codes
        want[2][b, :, o, 2 * i], want[2][b, :, o, 2 * i + 1] = sc, ze
        back.append(cc.values(codes, sc, ze).astype(np.float32))
    assert_cache((kc, vc, par), want)
    out = [torch.full((T, Hk, D), 5.0 + i, dtype=cc.TORCH[src], device=d) for i in range(2)]
    pa.paged_kv_read_int4(*out, torch.from_numpy(slots).to(d), kc, vc, par)
    for i, (got, v) in enumerate(zip(out, back)):
        ref = np.full((T, Hk, D), 5.0 + i, np.float32)
        ref[live] = v
        assert np.array_equal(got.float().cpu().numpy(), torch.from_numpy(ref).to(cc.TORCH[src]).float().numpy(),
                              equal_nan=True)
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT


def test_copy_blocks_moves_codes_and_parameters(pa):
    rng = np.random.default_rng(5)
    d = dev()
    NB, Hk, bs, D = 9, 3, 8, 64
    kc = torch.from_numpy(rng.integers(0, 256, (NB, Hk, bs, D // 2), dtype=np.uint8)).to(d)
    vc = torch.from_numpy(rng.integers(0, 256, (NB, Hk, bs, D // 2), dtype=np.uint8)).to(d)
    par = torch.from_numpy(rng.standard_normal((NB, Hk, bs, 4)).astype(np.float16)).to(d)
    want = [t.clone() for t in (kc, vc, par)]
    for s, t in ((0, 5), (7, 2)):
        for w in want:
            w[t] = w[s]
    pa.copy_blocks(kc, vc, torch.tensor([[0, 5], [7, 2]], dtype=torch.int32, device=d), kv_params=par)
    assert all(torch.equal(a, b) for a, b in zip((kc, vc, par), want))
    pa.copy_blocks(kc, vc, torch.tensor([[0, NB]], dtype=torch.int32, device=d), kv_params=par)
    assert pa.get_device_error() == pa.PA_DEVERR_COPY_PAIR


# ---------------------------------------------------------------------------- decode

class Case:
    """A paged 4-bit cache of random rows whose unused slots hold NaN parameters."""

    def __init__(self, rng, lens, H, Hk, D, bs, dtype, gain=1.0, k_size=1.0, v_size=1.0, reserve=0):
        self.lens, self.H, self.Hk, self.D, self.bs, self.dtype = np.asarray(lens, np.int32), H, Hk, D, bs, dtype
        self.bt, self.NB, _ = cc.tables(rng, lens, bs, reserve=reserve)
        self.kc = rng.integers(0, 256, (self.NB, Hk, bs, D // 2), dtype=np.uint8)
        self.vc = rng.integers(0, 256, (self.NB, Hk, bs, D // 2), dtype=np.uint8)
        self.par = np.full((self.NB, Hk, bs, 4), np.nan, np.float16)
        self.k, self.v = [], []
        for b, n in enumerate(self.lens):
            s = cc.slots_of(self.bt[b], n, bs)
            blk, off = s // bs, s % bs
            for x, cache, i, out in ((rows(rng, (n, Hk, D), "k") * k_size, self.kc, 0, self.k),
                                     (rows(rng, (n, Hk, D)) * v_size, self.vc, 2, self.v)):
                if n:
                    codes, sc, ze = cc.cache_rows(x.astype(np.float32))
                    cache[blk, :, off] = codes
                    self.par[blk, :, off, i] = sc
                    self.par[blk, :, off, i + 1] = ze
                    out.append(cc.values(codes, sc, ze))
                else:
                    out.append(np.zeros((0, Hk, D)))
        self.q = rng.standard_normal((len(lens), H, D)).astype(np.float32) * np.float32(gain)
        self.scale = D ** -0.5
        d = dev()
        self.t = {k: torch.from_numpy(v).to(d) for k, v in
                  (("kc", self.kc), ("vc", self.vc), ("par", self.par), ("bt", self.bt), ("lens", self.lens))}
        self.t["q"] = torch.from_numpy(self.q).to(d).to(cc.TORCH[dtype])

    def run(self, pa, mass=None, out=None, **kw):
        out = torch.full_like(self.t["q"], float("nan")) if out is None else out
        t = self.t
        pa.paged_attention_decode_int4(out, t["q"], t["kc"], t["vc"], t["par"], t["bt"], t["lens"], self.scale,
                                       mass=mass, **kw)
        return out

    def check(self, out, mass=None, before=0.0):
        got = out.double().cpu().numpy()
        qs = cc.stored(self.q, self.dtype)
        for b, n in enumerate(self.lens):
            ref, w, big, wv = cc.attention(qs[b], self.k[b], self.v[b], self.scale)
            dx = score_error(qs[b], self, b)
            tol = bound(ref, dx, parts(self, b, w), self.dtype)
            err = np.abs(got[b] - ref)
            assert np.isfinite(got[b]).all() and (err <= tol).all(), (b, n, float((err - tol).max()), float(err.max()))
            if mass is not None:
                m = mass[b].double().cpu().numpy()
                rel = 2 * dx + 8 * 2.0 ** -22
                mw = cc.group_mass(w, self.Hk)
                mt = cc.group_mass(w * (np.expm1(rel.max(1, initial=0.0))[:, None]), self.Hk)
                prior = before if np.isscalar(before) else before[b][:, :n]
                err = np.abs(m[:, :n] - mw - prior)
                # a weight below float32's least normal number, 2^-126, may be flushed to zero:
                # so may each of the up to 16 added up
                mt = mt + 16 * 2.0 ** -126
                assert (err <= mt + 2.0 ** -23 * (mw + np.abs(prior))).all(), (b, n, float((err - mt).max()))
                rest = m[:, n:]
                assert np.array_equal(rest, np.full_like(rest, before) if np.isscalar(before) else before[b][:, n:])


def score_error(q, case, b):
    """Bound on each score's error [H, n]: a sum of D + 2 products in float32, each product and
    partial sum off by at most 2^-23 of the absolute values summed -- of q times code * scale and
    of the zero times the sum of q, which the formula adds apart."""
    n = case.lens[b]
    s = cc.slots_of(case.bt[b], n, case.bs)
    blk, off = s // case.bs, s % case.bs
    G = case.H // case.Hk
    par = np.repeat(case.par[blk, :, off].astype(np.float64), G, 1)                 # [n, H, 4]
    codes = np.repeat(cc.unpack(case.kc[blk, :, off]).astype(np.float64), G, 1)    # [n, H, D]
    a = np.einsum("hd,nhd->hn", np.abs(q), codes) * np.abs(par[:, :, 0]).T
    a += np.abs(q).sum(1)[:, None] * np.abs(par[:, :, 1]).T
    return a * case.scale * (case.D + 2) * 2.0 ** -23


def parts(case, b, w):
    """Weighted sums of what an output is added up from, [H, D]: |code * v_scale| + |v_zero|. (Not
    of |v|: where code * scale and zero cancel, their roundings stay.)"""
    n = case.lens[b]
    s = cc.slots_of(case.bt[b], n, case.bs)
    blk, off = s // case.bs, s % case.bs
    par = np.abs(case.par[blk, :, off].astype(np.float64))                          # [n, Hk, 4]
    a = cc.unpack(case.vc[blk, :, off]) * par[:, :, 2, None] + par[:, :, 3, None]
    return np.einsum("hn,nhd->hd", w, np.repeat(a, case.H // case.Hk, 1))


def bound(ref, dx, a, dtype):
    """Output bound. Each term of an output's sum is off by its weight's error -- its own score's
    and the sum's, e^(2 dx) -- by 2^-11 (weights times V scales enter the products as f16) and by
    2^-20 (exp2, sums); the result is rounded once. A last term covers f16 subnormal outputs."""
    rel = np.expm1(2 * dx.max(1, initial=0.0)[:, None]) + 2.0 ** -11 + 2.0 ** -20
    return np.abs(ref) * cc.EPS[dtype] / 2 + (1 + cc.EPS[dtype]) * rel * a + cc.EPS[dtype] * 2.0 ** -14


RAGGED = [1, 7, 0, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300, 513, 1000, 1025]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hk,D,bs", [(8, 8, 128, 16), (32, 8, 128, 16), (6, 2, 64, 8), (7, 1, 128, 32), (16, 2, 64, 64),
                                       (12, 1, 128, 256), (32, 2, 128, 8), (10, 2, 64, 16),
                                       (16, 1, 64, 8), (3, 3, 64, 128)])
def test_decode_ragged(pa, dtype, H, Hk, D, bs):
    """Contexts of nothing, one token, tiles and their neighbours, several partitions; group
    sizes 1 to 16; from zero mass."""
    case = Case(np.random.default_rng(11 + H + D + bs), RAGGED, H, Hk, D, bs, dtype)
    mass = torch.zeros((len(RAGGED), Hk, 1030), device=dev())
    out = case.run(pa, mass, max_context_len=max(RAGGED))
    case.check(out, mass)
    assert pa.get_device_error() == 0
    plain = case.run(pa, max_context_len=max(RAGGED))
    assert torch.equal(out, plain)                       # accumulating weights does not change the output


@pytest.mark.parametrize("lens", [[2000, 1, 128, 700, 0, 1537], [31] * 700, [0, 0, 33], [0], [9000], [70, 5000] * 40])
@pytest.mark.parametrize("H,Hk", [(16, 4), (12, 1)])
def test_decode_cuts(pa, lens, H, Hk):
    """Rows that one run covers, rows cut into many, runs over many rows; non-zero mass."""
    case = Case(np.random.default_rng(3), lens, H, Hk, 128, 16, "f16")
    n = max(1, max(lens))
    mass = torch.full((len(lens), Hk, n), 0.25, device=dev())
    out = case.run(pa, mass, max_context_len=n)
    case.check(out, mass, before=0.25)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("gain,k_size,v_size", [(6.0, 1.0, 1.0), (1.0, 100.0, 1e-3), (1e-3, 1e-3, 1e-4), (300.0, 0.01, 2e3)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_ranges(pa, dtype, gain, k_size, v_size):
    """Peaked and flat softmaxes; caches of large and of tiny values (parameters down to f16
    subnormals), queries of large and of tiny ones."""
    case = Case(np.random.default_rng(21), [400, 90], 8, 2, 128, 16, dtype, gain, k_size, v_size)
    mass = torch.zeros((2, 2, 400), device=dev())
    case.check(case.run(pa, mass), mass)


def test_decode_one_dominant_token(pa):
    """A first token that takes nearly all the weight of long flat contexts, and small V rows next
    to large ones: the many light tokens still count."""
    case = Case(np.random.default_rng(23), [3000, 2500], 8, 2, 128, 16, "f16", gain=0.1)
    qs = cc.stored(case.q, "f16")
    for b in range(2):
        for h in range(2):
            d = np.sign(qs[b, 4 * h:4 * h + 4].sum(0)).astype(np.float32) * 40.0
            codes, s, z = cc.cache_rows(d)
            blk = case.bt[b, 0]
            case.kc[blk, h, 0], case.par[blk, h, 0, 0], case.par[blk, h, 0, 1] = codes, s, z
            case.k[b][0, h] = cc.values(codes, s, z)
            codes, s, z = cc.cache_rows(np.linspace(-50, 50, 128).astype(np.float32))
            case.vc[blk, h, 0], case.par[blk, h, 0, 2], case.par[blk, h, 0, 3] = codes, s, z
            case.v[b][0, h] = cc.values(codes, s, z)
    for k in ("kc", "vc", "par"):
        case.t[k] = torch.from_numpy(getattr(case, k)).to(dev())
    mass = torch.zeros((2, 2, 3000), device=dev())
    case.check(case.run(pa, mass), mass)


def test_decode_long_context(pa):
    case = Case(np.random.default_rng(31), [20011, 6], 8, 1, 128, 16, "bf16", gain=2.0)
    mass = torch.zeros((2, 1, 20011), device=dev())
    case.check(case.run(pa, mass), mass)


def test_decode_many_sequences(pa):
    """More sequences than one launch takes."""
    rng = np.random.default_rng(41)
    lens = rng.integers(0, 40, 3500)
    case = Case(rng, lens, 4, 2, 64, 8, "bf16")
    mass = torch.zeros((3500, 2, 40), device=dev())
    case.check(case.run(pa, mass, max_context_len=40), mass)
    assert pa.get_device_error() == 0


def test_decode_repeats_bit_for_bit_and_leaves_inputs(pa):
    case = Case(np.random.default_rng(51), [777, 64, 1300], 32, 8, 128, 16, "bf16")
    before = {k: v.clone() for k, v in case.t.items()}
    m0 = torch.zeros((3, 8, 1300), device=dev())
    first = case.run(pa, m0)
    for _ in range(3):
        m = torch.zeros_like(m0)
        assert torch.equal(case.run(pa, m), first) and torch.equal(m, m0)
    for k, v in before.items():
        assert torch.equal(v.view(torch.uint8), case.t[k].view(torch.uint8))


def test_decode_nan_parameter_inside_a_context(pa):
    case = Case(np.random.default_rng(61), [200, 200], 8, 2, 128, 16, "bf16")
    good = case.run(pa)
    case.t["par"][int(case.bt[1, 3]), 1, 5, 0] = float("nan")
    out = case.run(pa)
    assert torch.equal(out[0], good[0]) and torch.equal(out[1, :4], good[1, :4])
    assert torch.isnan(out[1, 4:].float()).all()


def test_decode_device_errors(pa):
    """Bad table entries read as zeros; lengths out of range are cut; both are reported."""
    case = Case(np.random.default_rng(71), [100, 60], 8, 2, 128, 16, "bf16")
    case.t["bt"][0, 2] = case.NB + 5
    out = case.run(pa)
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
    case.k[0][32:48] = 0.0
    case.v[0][32:48] = 0.0
    par = case.par.copy()
    got = out.double().cpu().numpy()
    qs = cc.stored(case.q, "bf16")
    ref, w, _, wv = cc.attention(qs[0], case.k[0], case.v[0], case.scale)
    assert (np.abs(got[0] - ref) <= np.abs(ref) * 2.0 ** -8 + 0.02 * wv).all()
    assert np.isfinite(got).all() and par.shape == case.par.shape
    case = Case(np.random.default_rng(72), [100, 60], 8, 2, 128, 16, "bf16")
    full = case.run(pa)
    case.t["lens"][1] = -3
    out = case.run(pa)
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT
    assert torch.equal(out[0], full[0]) and (out[1] == 0).all()
    case.t["lens"][1] = 60
    mass = torch.zeros((2, 2, 64), device=dev())
    out = case.run(pa, mass)                           # a context longer than mass holds
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT
    case.lens = np.array([64, 60], np.int32)
    case.k[0], case.v[0] = case.k[0][:64], case.v[0][:64]
    case.check(out, mass)


def test_decode_workspaces_and_streams(pa):
    """A caller's workspace, too small a one, none through the C ABI; another stream."""
    case = Case(np.random.default_rng(81), [1500, 1400], 8, 2, 128, 16, "f16")
    want_mass = torch.zeros((2, 2, 1500), device=dev())
    want = case.run(pa, want_mass)
    need = pa.decode_int4_workspace_bytes(2, 8, 2, 128, case.bt.shape[1] * 16, True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev())
    mass = torch.zeros_like(want_mass)
    assert torch.equal(case.run(pa, mass, workspace=ws), want) and torch.equal(mass, want_mass)
    with pytest.raises(pa.PagedAttnError) as e:
        case.run(pa, mass, workspace=ws[:need - 16])
    assert e.value.status == pa.PA_ERR_WORKSPACE
    t, out, mass = case.t, torch.empty_like(want), torch.zeros_like(want_mass)
    rc = pa.lib().pa_paged_attention_decode_int4(
        out.data_ptr(), t["q"].data_ptr(), t["kc"].data_ptr(), t["vc"].data_ptr(), t["par"].data_ptr(),
        mass.data_ptr(), 1500, t["bt"].data_ptr(), case.bt.shape[1], t["lens"].data_ptr(), 2, 8, 2, 128, 16, case.NB,
        case.scale, 0, None, 0, pa.PA_DTYPE_F16, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(out, want) and torch.equal(mass, want_mass)
    side = torch.cuda.Stream()
    mass = torch.zeros_like(want_mass)
    torch.cuda.synchronize()
    out = case.run(pa, mass, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(mass, want_mass)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [500, 20000])
def test_decode_error_of_flat_contexts(pa, n, D):
    """The rounding of the weights must not be amplified by what cancels between codes and zeros.

    f16 weights are off by at most half a step, 2^-11 of their power of two: 2^-11 / sqrt(3) = 2.8e-4 in
    the root mean square at most, independently of each other. Each is multiplied by a value about the
    row's middle, so the output's relative error is 2.8e-4 times that value's size against the values'
    own (1 for rows that are symmetric; 1.05 allowed), and the output's own rounding adds as much:
    sqrt(2.8e-4^2 * 1.05^2 + 2.8e-4^2) = 4.1e-4. (The products of plain codes with the weights are off
    by 1.9 times as much: 6.1e-4.) The norms are over 2048 outputs or more: 5 % of scatter at most."""
    rng = np.random.default_rng(n + D)
    case = Case(rng, [n, n], 8, 2, D, 16, "f16")
    t = case.t
    k, v = (torch.from_numpy(rng.standard_normal((2 * n, 2, D)).astype(np.float32)).to(dev()) for _ in range(2))
    slots = torch.from_numpy(np.concatenate([case.bt[b][np.arange(n) // 16] * 16 + np.arange(n) % 16
                                             for b in range(2)]).astype(np.int32)).to(dev())
    pa.paged_kv_write_int4(k, v, slots, t["kc"], t["vc"], t["par"])
    hk, hv = torch.empty_like(k), torch.empty_like(v)
    pa.paged_kv_read_int4(hk, hv, slots, t["kc"], t["vc"], t["par"])
    q = torch.from_numpy(rng.standard_normal((2, 8, D)).astype(np.float32)).to(dev()).half()
    out = torch.empty_like(q)
    pa.paged_attention_decode_int4(out, q, t["kc"], t["vc"], t["par"], t["bt"], t["lens"], D ** -0.5)
    hk, hv = (x.double().view(2, n, 2, D) for x in (hk, hv))
    w = torch.softmax(torch.einsum("bhgd,bthd->bhgt", q.double().view(2, 2, 4, D), hk) * D ** -0.5, -1)
    ref = torch.einsum("bhgt,bthd->bhgd", w, hv).reshape(2, 8, D)
    err = float((out.double() - ref).norm() / ref.norm())
    assert err <= 4.1e-4 * 1.05, err
