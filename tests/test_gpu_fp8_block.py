"""The block-scaled 8-bit cache on the GPU against plain 64-bit forms: scatter, read-back and copies
bit for bit, decode within a bound that follows from its roundings (see bound())."""
import numpy as np
import pytest
import torch

import compress_cases as cc
import step_cases as sc
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

class Store:
    """A cache on the device and its plain double, at first with codes of anything and no valid scale."""

    def __init__(self, NB, Hk, bs, D, seed=0, scales=np.nan):
        rng = np.random.default_rng(seed)
        self.kc, self.vc = (rng.integers(0, 256, (NB, Hk, bs, D), dtype=np.uint8) for _ in range(2))
        self.sc = np.full((NB, Hk, 2), scales, np.float32)
        self.t = [torch.from_numpy(x).to(dev()) for x in (self.kc, self.vc, self.sc)]

    def write(self, pa, k, v, slots, src, kt=None, vt=None):
        kt = torch.from_numpy(k).to(dev()).to(cc.TORCH[src]) if kt is None else kt
        vt = torch.from_numpy(v).to(dev()).to(cc.TORCH[src]) if vt is None else vt
        pa.paged_kv_write_fp8_block(kt, vt, torch.as_tensor(np.asarray(slots, np.int32), device=dev()), *self.t)
        sc.write_blocks(self.kc, self.vc, self.sc, cc.stored(k, src), cc.stored(v, src), slots)

    def check(self):
        for t, w in zip(self.t[:2], (self.kc, self.vc)):
            assert sc.same_codes(t.cpu().numpy(), w)
        assert np.array_equal(self.t[2].cpu().numpy(), self.sc, equal_nan=True)


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hk,D,bs", [(1, 128, 16), (8, 128, 16), (3, 64, 8), (5, 64, 256), (2, 128, 64)])
def test_write_is_bit_exact(pa, src, Hk, D, bs):
    """Sequences that grow by chunks and single tokens, some far larger than what their blocks held:
    new blocks, blocks whose scale grows, blocks filled across calls, padding."""
    rng = np.random.default_rng(7 + D + bs)
    lens = [0, 5, 0, 2 * bs + 1]
    total = [3 * bs + 7] * 4
    bt, NB, _ = cc.tables(rng, total, bs)
    s = Store(NB, Hk, bs, D)
    at = [0] * 4
    for step in range(7):
        slots, big = [], []
        for b in range(4):
            n = (lens[b], 1, bs + 3, 1, 2, 0, 1)[step]
            n = min(n, total[b] - at[b])
            slots += list(cc.slots_of(bt[b], total[b], bs)[at[b]:at[b] + n])
            at[b] += n
        slots = [-1] * (step == 3) + slots + [-1] * (step % 3)
        T = len(slots)
        big = np.where(rng.random((T, 1, 1)) < 0.3, np.float32(30.0), np.float32(1.0)).astype(np.float32)
        s.write(pa, rows(rng, (T, Hk, D), "k") * big, rows(rng, (T, Hk, D)) * big[::-1].copy(), slots, src)
        s.check()
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("T,Hk,D,bs", [(31, 5, 128, 16), (33, 8, 64, 8), (65, 3, 64, 32), (200, 1, 128, 16), (700, 2, 128, 64),
                                       (1000, 7, 64, 256), (6000, 1, 64, 8)])
def test_write_and_read_mixed_batches(pa, T, Hk, D, bs):
    """Single tokens, runs of a few and of more than a block, side by side, between them tokens without a slot and
    with a bad one; read back at once, and again a call later."""
    rng = np.random.default_rng(T + Hk + bs)
    total = 4 * bs
    bt, NB, _ = cc.tables(rng, [total] * T, bs)
    s, at = Store(NB, Hk, bs, D), np.zeros(T, int)
    for call in range(2):
        slots, bad = [], 0
        for b in rng.permutation(T):
            n = int(rng.choice([1, 1, 1, 1, 2, 3, 17, 40, bs + 5]))
            n = min(n, total - at[b], T - len(slots))
            slots += list(cc.slots_of(bt[b], total, bs)[at[b]:at[b] + n])
            at[b] += n
            if rng.random() < 0.2 and len(slots) < T:
                slots.append(-1 if rng.random() < 0.7 else NB * bs + int(rng.integers(0, 9)))
                bad += slots[-1] >= 0
            if len(slots) >= T:
                break
        slots = np.asarray(slots[:T], np.int32)
        big = np.where(rng.random((T, 1, 1)) < 0.3, np.float32(30.0), np.float32(1.0)).astype(np.float32)
        good = np.where(slots < NB * bs, slots, -1)
        k, v = rows(rng, (T, Hk, D), "k") * big, rows(rng, (T, Hk, D)) * big
        kt, vt = (torch.from_numpy(x).to(dev()).to(torch.bfloat16) for x in (k, v))
        st = torch.from_numpy(slots).to(dev())
        pa.paged_kv_write_fp8_block(kt, vt, st, *s.t)
        ko, vo = (torch.full((T, Hk, D), 7.0, device=dev()) for _ in range(2))
        pa.paged_kv_read_fp8_block(ko, vo, st, *s.t)
        sc.write_blocks(s.kc, s.vc, s.sc, cc.stored(k, "bf16"), cc.stored(v, "bf16"), good)
        s.check()
        blk, off = good // bs, good % bs
        for got, cache, i in ((ko, s.kc, 0), (vo, s.vc, 1)):
            want = np.where((good >= 0)[:, None, None], sc.E4M3[cache[blk, :, off]] * s.sc[blk, :, i][..., None].astype(np.float64), 7.0)
            assert np.array_equal(got.double().cpu().numpy(), want)          # a code times a power of two: exact
        assert pa.get_device_error() == (pa.PA_DEVERR_SLOT if bad else 0)


@pytest.mark.parametrize("bs", [8, 32])
def test_write_order_within_a_block(pa, bs):
    """The tokens of a block next to each other, in any order; the first slot last."""
    rng = np.random.default_rng(3)
    s = Store(5, 2, bs, 64)
    order = [rng.permutation(bs) + b * bs for b in (3, 0, 4)]
    order[1] = order[1][order[1] != 0][:bs - 2]                   # a block never started: its scales are no numbers
    slots = np.concatenate(order)
    s.write(pa, rows(rng, (len(slots), 2, 64), "k"), rows(rng, (len(slots), 2, 64)), slots, "f32")
    s.check()


def test_write_special_values(pa):
    """Zeros, tiny, huge, infinite and NaN elements, exact ties, values at the border of a scale, scales that
    are no powers of two, zero, negative or infinite."""
    D, bs = 128, 8
    base = np.linspace(-3.0, 4.5, D).astype(np.float32)
    ties = ((np.arange(D) % 16 + 0.5) / 8 * np.exp2(np.arange(D) // 16 - 4.0)).astype(np.float32)
    r = [np.zeros(D), np.full(D, -0.0), base * 1e-38, base * 1e-44, base * 1e30, np.full(D, 3.4e38),
         np.where(np.arange(D) == 5, np.inf, base), np.where(np.arange(D) == 9, -np.inf, base),
         np.where(np.arange(D) == 77, np.nan, base), np.full(D, np.nan), np.full(D, np.inf), ties,
         np.where(np.arange(D) == 3, 448.0, base), np.where(np.arange(D) == 3, np.nextafter(np.float32(448), np.float32(500)), base)]
    x = np.stack(r).astype(np.float32)[:, None, :]
    s = Store(len(r), 1, bs, D)
    s.write(pa, x, x[::-1].copy(), np.arange(len(r)) * bs, "f32")          # each starts a block
    s.check()
    s.write(pa, x[::-1].copy(), x, np.arange(len(r)) * bs + 1, "f32")      # each joins one
    s.check()
    for i, scale in enumerate([0.3, 0.0, -1.0, np.inf, np.nan, 1e-42, 3e38, 2.0 ** -126]):
        s = Store(2, 1, bs, D, seed=i, scales=scale)
        for j, m in enumerate((1.0, 1000.0)):
            y = base[None, None, :] * np.float32(m)
            s.write(pa, y, y, [3 + j], "f32")
            s.check()
    assert pa.get_device_error() == 0


def test_write_strided_rows_and_errors(pa):
    """k and v as views of a fused projection; slots out of range."""
    rng = np.random.default_rng(5)
    T, H, Hk, D, bs = 19, 3, 2, 64, 8
    x = torch.from_numpy(rows(rng, (T, H + 2 * Hk, D))).to(dev()).bfloat16()
    k, v = x[:, H:H + Hk], x[:, H + Hk:]
    slots = list(range(8, 16)) + [-1, 40, -7] + list(range(24, 32))
    s = Store(5, Hk, bs, D)
    s.write(pa, k.float().cpu().numpy(), v.float().cpu().numpy(), slots, "bf16", k, v)
    s.check()
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT
    one = k[:1].expand(T, Hk, D)                                           # the same row for every token
    s.write(pa, one.float().cpu().numpy(), v.float().cpu().numpy(), slots, "bf16", one, v)
    s.check()
    with pytest.raises(ValueError, match="heads of a token"):
        pa.paged_kv_write_fp8_block(x[:, :2 * Hk:2], v, torch.zeros(T, dtype=torch.int32, device=dev()), *s.t)
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT


@pytest.mark.parametrize("dst", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hk,D,bs", [(1, 1, 128, 16), (53, 8, 128, 32), (5501, 3, 64, 8), (4000, 2, 128, 256)])
def test_read_back(pa, dst, T, Hk, D, bs):
    """Repeated slots, -1 and out-of-range ones; rows of those stay as they were."""
    rng = np.random.default_rng(70 + T)
    NB = 6
    s = Store(NB, Hk, bs, D, seed=T)
    s.sc[:] = rng.choice([1.0, 0.25, 2.0 ** -20, 0.3, 7.7], s.sc.shape)
    s.t[2].copy_(torch.from_numpy(s.sc))
    slots = rng.integers(0, NB * bs, T).astype(np.int32)
    if T > 8:
        slots[3], slots[5], slots[7] = -1, NB * bs, -9
    out = [torch.full((T, Hk, D), 5.0 + i, dtype=cc.TORCH[dst], device=dev()) for i in range(2)]
    pa.paged_kv_read_fp8_block(*out, torch.from_numpy(slots).to(dev()), *s.t)
    assert pa.get_device_error() == (pa.PA_DEVERR_SLOT if T > 8 else 0)
    live = (slots >= 0) & (slots < NB * bs)
    for i, (o, c) in enumerate(zip(out, (s.kc, s.vc))):
        ref = np.full((T, Hk, D), 5.0 + i, np.float32)
        ref[live] = sc.block_values(c, s.sc, i)[slots[live] // bs, :, slots[live] % bs].astype(np.float32)
        want = torch.from_numpy(ref).to(cc.TORCH[dst])
        assert np.array_equal(o.float().cpu().numpy(), want.float().numpy(), equal_nan=True)


def test_copy_blocks_moves_codes_and_scales(pa):
    s = Store(9, 3, 8, 64, seed=2, scales=1.0)
    s.t[2].copy_(torch.arange(54, device=dev()).view(9, 3, 2))
    want = [t.clone() for t in s.t]
    for a, b in ((0, 5), (7, 2)):
        for w in want:
            w[b] = w[a]
    pa.copy_blocks(*s.t[:2], torch.tensor([[0, 5], [7, 2]], dtype=torch.int32, device=dev()), kv_scales=s.t[2])
    assert all(torch.equal(a, b) for a, b in zip(s.t, want))
    pa.copy_blocks(*s.t[:2], torch.tensor([[0, 9], [-1, 2]], dtype=torch.int32, device=dev()), kv_scales=s.t[2])
    assert all(torch.equal(a, b) for a, b in zip(s.t, want))
    assert pa.get_device_error() == pa.PA_DEVERR_COPY_PAIR


# ---------------------------------------------------------------------------- decode

class Case:
    """A paged cache of random rows. Codes of NaN lie past every context's end, NaN scales in the blocks
    that no context has."""

    def __init__(self, rng, lens, H, Hk, D, bs, dtype, gain=1.0, k_size=1.0, v_size=1.0, spread=1.0, reserve=0):
        self.lens, self.H, self.Hk, self.D, self.bs, self.dtype = np.asarray(lens, np.int32), H, Hk, D, bs, dtype
        self.bt, self.NB, _ = cc.tables(rng, lens, bs, reserve=reserve)
        self.kc, self.vc = (np.full((self.NB, Hk, bs, D), c, np.uint8) for c in (0x7F, 0xFF))
        self.sc = np.full((self.NB, Hk, 2), np.nan, np.float32)
        for b, n in enumerate(self.lens):
            for j in range(-(-int(n) // bs)):
                blk, m = self.bt[b, j], min(bs, int(n) - j * bs)
                for i, (c, size) in enumerate(((self.kc, k_size), (self.vc, v_size))):
                    # neighbouring blocks of unlike size
                    x = rows(rng, (Hk, m, D), "k" if i == 0 else "plain") * size * spread ** rng.uniform(-1, 1)
                    for h in range(Hk):
                        s = sc.scale_for(np.abs(x[h]).max())
                        self.sc[blk, h, i] = s
                        c[blk, h, :m] = sc.encode(x[h].astype(np.float64) / s)
        self.q = rng.standard_normal((len(lens), H, D)).astype(np.float32) * np.float32(gain)
        self.scale = D ** -0.5
        self.t = {k: torch.from_numpy(v).to(dev()) for k, v in
                  (("kc", self.kc), ("vc", self.vc), ("sc", self.sc), ("bt", self.bt), ("lens", self.lens))}
        self.t["q"] = torch.from_numpy(self.q).to(dev()).to(cc.TORCH[dtype])

    def kv(self, b):
        """float64 K and V [n, Hk, D] of sequence b."""
        n = int(self.lens[b])
        t = np.arange(n)
        blk, off = self.bt[b, t // self.bs], t % self.bs
        return [sc.E4M3[c[blk, :, off]] * self.sc[blk, :, i].astype(np.float64)[..., None]
                for i, c in enumerate((self.kc, self.vc))]

    def run(self, pa, out=None, **kw):
        out = torch.full_like(self.t["q"], float("nan")) if out is None else out
        t = self.t
        pa.paged_attention_decode_fp8_block(out, t["q"], t["kc"], t["vc"], t["sc"], t["bt"], t["lens"], self.scale, **kw)
        return out

    def check(self, out):
        got = out.double().cpu().numpy()
        qs = cc.stored(self.q, self.dtype)
        for b, n in enumerate(self.lens):
            ref, tol = expected(qs[b], *self.kv(b), self.scale, self.dtype)
            with np.errstate(invalid="ignore"):
                err = np.abs(got[b] - ref)
            # f16 ends at 65504: what rounds past it, 65520 and beyond, is infinite
            top = 65520.0 if self.dtype == "f16" else np.inf
            inf = np.isinf(got[b]) & (np.sign(got[b]) == np.sign(ref)) & (np.abs(ref) + tol >= top)
            assert (inf | (np.isfinite(got[b]) & (err <= tol))).all(), (b, n, float((err - tol).max()), float(err.max()))


def expected(q, k, v, scale, dtype):
    """(output, bound) of one sequence. A score is a sum of D products in float32, each product and
    partial sum off by at most 2^-23 of the absolute values summed, two more for the scales; the query's
    channels enter as f16 times a power of two, within 2^-36 of the row's largest. Each term of an
    output's sum is off by its weight's error -- its own score's and the sum's, e^(2 dx) --, by 2^-11
    (weights times V scales enter the products as f16) and by 2^-20 (exp2, sums); below 2^-22 of the largest
    weight times the largest V scale (at most twice the largest |V| over 448, where a code may be 448) they are
    within 2^-33 of that. The result is rounded once, in f16 to multiples of 2^-24."""
    n = k.shape[0]
    ref, w, big, wv = cc.attention(q, k, v, scale)
    dx = big * (q.shape[1] + 4) * 2.0 ** -23
    if n:
        G = q.shape[0] // k.shape[1]
        dx = dx + abs(scale) * 2.0 ** -36 * np.abs(q).max(1)[:, None] * np.repeat(np.abs(k).sum(2).T, G, 0)
    rel = np.expm1(2 * dx.max(1, initial=0.0)[:, None]) + 2.0 ** -11 + 2.0 ** -20
    # a V scale is at most 2^-100 or, as the power of two that the scatter takes, 2 |V| / 448
    eps, small = cc.EPS[dtype], n * 2.0 ** -33 * 448 * 2 * max(2 * np.abs(v).max(initial=0.0) / 448, 2.0 ** -100)
    return ref, np.abs(ref) * eps / 2 + (1 + eps) * (rel * wv + small) + eps * 2.0 ** -14


RUNS = 100000                                # a bound on the contexts at which any call is cut into runs

RAGGED = [1, 7, 0, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300, 513, 1000, 1025]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hk,D,bs", [(8, 8, 128, 16), (32, 8, 128, 16), (6, 2, 64, 8), (7, 1, 128, 32), (16, 2, 64, 64),
                                       (12, 1, 128, 256), (32, 2, 128, 8), (10, 2, 64, 16),
                                       (16, 1, 64, 8), (3, 3, 64, 128)])
def test_decode_ragged(pa, dtype, H, Hk, D, bs):
    """Contexts of nothing, one token, stages and their neighbours, many runs; groups of 1 to 16."""
    case = Case(np.random.default_rng(11 + H + D + bs), RAGGED, H, Hk, D, bs, dtype)
    out = case.run(pa, max_context_len=max(RAGGED))
    case.check(out)
    assert torch.equal(out, case.run(pa, max_context_len=max(RAGGED)))
    case.check(case.run(pa))
    case.check(case.run(pa, max_context_len=RUNS))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("lens", [[2000, 1, 128, 700, 0, 1537], [31] * 700, [0, 0, 33], [0], [9000], [5000], [4000, 2100, 0, 1], [70, 5000] * 20,
                                  [5] * 1600])
@pytest.mark.parametrize("H,Hk", [(16, 4), (12, 1)])
def test_decode_cuts(pa, lens, H, Hk):
    """Rows that one run covers, rows cut into many, runs over many rows, batches of several launches."""
    case = Case(np.random.default_rng(3), lens, H, Hk, 128, 16, "f16")
    for bound in (max(1, max(lens)), RUNS):
        case.check(case.run(pa, max_context_len=bound))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("gain,k_size,v_size,spread", [(6.0, 1.0, 1.0, 1.0), (1.0, 100.0, 1e-3, 4.0), (1e-3, 1e-3, 1e-4, 1.0),
                                                       (300.0, 0.01, 2e3, 30.0), (1e4, 1e-6, 1.0, 1e3)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_ranges(pa, dtype, gain, k_size, v_size, spread, D):
    """Peaked and flat softmaxes; caches and queries of large and of tiny values; blocks of unlike size."""
    case = Case(np.random.default_rng(21), [400, 90], 8, 2, D, 16, dtype, gain, k_size, v_size, spread)
    case.check(case.run(pa))
    case.check(case.run(pa, max_context_len=RUNS))


@pytest.mark.parametrize("D", [64, 128])
def test_decode_v_blocks_far_apart(pa, D):
    """One block of V 2^30 times the others, its keys of little weight; and scales down to 2^-100."""
    case = Case(np.random.default_rng(23), [300, 300], 8, 2, D, 16, "bf16", gain=2.0)
    case.sc[case.bt[0, 5], :, 1] *= np.float32(2.0 ** 30)
    case.sc[case.bt[1, :19], :, 1] = np.float32(2.0 ** -100)
    case.t["sc"].copy_(torch.from_numpy(case.sc))
    case.check(case.run(pa))
    case.check(case.run(pa, max_context_len=RUNS))


@pytest.mark.parametrize("bound", [0, RUNS])
def test_decode_nan_and_bad_blocks(pa, bound):
    """A NaN code of K or V, or a NaN scale, reaches the outputs of its kv head and no other's; bad block
    ids read as zeros."""
    case = Case(np.random.default_rng(29), [100, 60, 100, 70], 8, 2, 128, 16, "bf16")
    want = case.run(pa, max_context_len=bound).clone()
    case.t["kc"][int(case.bt[0, 2]), 1, 3, 77] = 0x7F
    case.t["vc"][int(case.bt[1, 1]), 0, 9, 5] = 0xFF
    case.t["sc"][int(case.bt[2, 0]), 1, 1] = float("nan")
    out = case.run(pa, max_context_len=bound)
    assert torch.isnan(out[0, 4:]).all() and torch.equal(out[0, :4], want[0, :4])
    assert torch.isnan(out[1, :4, 5]).all() and torch.equal(out[1, 4:], want[1, 4:])
    assert torch.isnan(out[2, 4:]).all() and torch.equal(out[2, :4], want[2, :4])
    assert torch.equal(out[3], want[3]) and pa.get_device_error() == 0
    for i, bad in ((0, case.NB), (4, -1), (3, 1 << 30)):
        b = case.bt[3, i]
        case.t["bt"][3, i] = bad
        case.kc[b], case.vc[b], case.sc[b] = 0, 0, 1.0
        out = case.run(pa, max_context_len=bound)
        assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
        ref, tol = expected(cc.stored(case.q, "bf16")[3], *case.kv(3), case.scale, "bf16")
        assert (np.abs(out[3].double().cpu().numpy() - ref) <= tol).all()


def test_decode_bad_lengths(pa):
    """Negative lengths count as none, lengths past the table or the bound as what these hold."""
    case = Case(np.random.default_rng(31), [100, 60, 90], 8, 2, 64, 16, "f16")
    want = case.run(pa)
    case.t["lens"].copy_(torch.tensor([-3, 60, 200], dtype=torch.int32))
    out = case.run(pa, max_context_len=90)
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT
    assert (out[0] == 0).all() and torch.equal(out[1], want[1])
    got, ref = out[2].double().cpu().numpy(), want[2].double().cpu().numpy()
    assert np.abs(got - ref).max() <= 2e-3                # the same context, in other runs


@pytest.mark.parametrize("bound", [0, RUNS])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn])
def test_decode_workspaces_and_cache_types(pa, dtype, bound):
    case = Case(np.random.default_rng(37), [700, 1500], 16, 4, 128, 32, "bf16")
    want = case.run(pa, max_context_len=bound)
    case.t["kc"], case.t["vc"] = case.t["kc"].view(dtype), case.t["vc"].view(dtype)
    n = pa.decode_fp8_block_workspace_bytes(2, 16, 4, 128, bound or case.bt.shape[1] * 32)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev())
        assert torch.equal(case.run(pa, workspace=ws, max_context_len=bound), want)
    with pytest.raises(pa.PagedAttnError) as e:
        case.run(pa, workspace=ws[:n - 16], max_context_len=bound)
    assert e.value.status == pa.PA_ERR_WORKSPACE
    # NULL: the library's own
    t, out = case.t, torch.empty_like(want)
    rc = pa.lib().pa_paged_attention_decode_fp8_block(
        out.data_ptr(), t["q"].data_ptr(), t["kc"].data_ptr(), t["vc"].data_ptr(), t["sc"].data_ptr(), t["bt"].data_ptr(),
        case.bt.shape[1], t["lens"].data_ptr(), 2, 16, 4, 128, 32, case.NB, case.scale, bound, None, 0, pa.PA_DTYPE_BF16,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(out, want)


def test_offsets_past_32_bits(pa):
    """Blocks at the far end of caches of more than 4 GiB, written, read and attended."""
    rng = np.random.default_rng(41)
    Hk, bs, D, H, NB, n = 8, 64, 128, 16, 68000, 150
    kc = torch.empty((NB, Hk, bs, D), dtype=torch.uint8, device=dev())
    vc, s = torch.empty_like(kc), torch.full((NB, Hk, 2), float("nan"), device=dev())
    assert kc.numel() > 1 << 32
    bt = np.array([[NB - 1, 3, NB - 7]], np.int32)
    slots = torch.from_numpy(cc.slots_of(bt[0], n, bs).astype(np.int32)).to(dev())
    k, v = (torch.from_numpy(rows(rng, (n, Hk, D))).to(dev()).bfloat16() for _ in range(2))
    pa.paged_kv_write_fp8_block(k, v, slots, kc, vc, s)
    back = [torch.empty((n, Hk, D), device=dev()) for _ in range(2)]
    pa.paged_kv_read_fp8_block(*back, slots, kc, vc, s)
    hk, hv = (x.double().cpu().numpy() for x in back)
    for x, h in ((k, hk), (v, hv)):                       # an E4M3's rounding: 2^-4, or half of 2^-9 scales
        x = x.double().cpu().numpy()
        assert (np.abs(x - h) <= np.abs(x) * 2.0 ** -4 + np.abs(x).max() / 224 * 2.0 ** -10).all()
    q = torch.from_numpy(rng.standard_normal((1, H, D)).astype(np.float32)).to(dev()).half()
    out = torch.empty_like(q)
    pa.paged_attention_decode_fp8_block(out, q, kc, vc, s, torch.from_numpy(bt).to(dev()),
                                        torch.tensor([n], dtype=torch.int32, device=dev()), D ** -0.5)
    ref, tol = expected(q[0].double().cpu().numpy(), hk, hv, D ** -0.5, "f16")
    assert (np.abs(out[0].double().cpu().numpy() - ref) <= tol).all()
    assert pa.get_device_error() == 0


SHORT = [1, 7, 0, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300, 513, 1000, 1024]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hk,D,bs", [(8, 8, 128, 16), (36, 9, 128, 16), (6, 2, 64, 8), (7, 1, 128, 32), (16, 2, 64, 64),
                                       (12, 1, 128, 256), (32, 2, 128, 8), (10, 2, 64, 16), (16, 1, 64, 8),
                                       (3, 3, 64, 128), (24, 4, 128, 16), (9, 3, 64, 32)])
def test_decode_rows_of_ctas(pa, dtype, H, Hk, D, bs):
    """Few rows of short contexts, which clusters of one to sixteen CTAs take: CTAs and warps without a stage, parts of a
    stage, several; the same contexts under a longer bound, which are cut into runs."""
    case = Case(np.random.default_rng(43 + H + D + bs), SHORT, H, Hk, D, bs, dtype, gain=2.0)
    out = case.run(pa, max_context_len=1024)
    case.check(out)
    assert torch.equal(out, case.run(pa, max_context_len=1024))
    case.check(case.run(pa, max_context_len=9000))
    case.check(case.run(pa, max_context_len=40000))
    assert (out[2] == 0).all() and pa.get_device_error() == 0
    # NaN in one row's context, a bad block and bad lengths in others
    want = out.clone()
    case.t["kc"][int(case.bt[15, 0]), 0, 3, 9] = 0x7F
    case.t["bt"][14, 1] = case.NB
    case.t["lens"][:2] = torch.tensor([-1, 5000], dtype=torch.int32)
    out = case.run(pa, max_context_len=1024)
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID | pa.PA_DEVERR_CONTEXT
    G = H // Hk
    assert torch.isnan(out[15, :G]).all() and torch.equal(out[15, G:], want[15, G:])
    assert (out[0] == 0).all() and torch.isfinite(out[14]).all() and torch.equal(out[3:14], want[3:14])
