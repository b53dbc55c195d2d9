"""Eviction by accumulated attention weight: what stays, where it moves and what is left
alone, against a host sort, bit for bit; a serving run of scored steps and evictions."""
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


def masses(rng, shape, kind):
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32) * np.float32(0.25)
    if kind == "equal":
        return np.full(shape, 0.125, np.float32)
    if kind == "crowd":                      # one exponent and two mantissa bits for all but a few
        return (1.0 + 0.2 * rng.random(shape)).astype(np.float32)
    m = rng.random(shape).astype(np.float32) ** 8
    if kind == "special":
        flat = m.reshape(-1)
        at = rng.permutation(flat.size)
        q = flat.size // 8
        flat[at[:q]] = np.nan
        flat[at[q:2 * q]] = np.inf
        flat[at[2 * q:3 * q]] = 0.0
        flat[at[3 * q:4 * q]] = -0.0
        flat[at[4 * q:5 * q]] = -flat[at[4 * q:5 * q]]
        flat[at[5 * q:6 * q]] = 1e-42
    return m


def caches(rng, NB, bs, Hk, D, dtype):
    if dtype == "int4":
        kc = rng.integers(0, 256, (NB, Hk, bs, D // 2), dtype=np.uint8)
        par = rng.standard_normal((NB, Hk, bs, 4)).astype(np.float16)
        return kc, rng.integers(0, 256, kc.shape, dtype=np.uint8), par
    if dtype == "e4m3":
        kc = rng.integers(0, 256, (NB, bs, Hk, D), dtype=np.uint8)
        return kc, rng.integers(0, 256, kc.shape, dtype=np.uint8), None
    e = np.uint32 if dtype == "f32" else np.uint16           # any bits: rows move unchanged
    kc = rng.integers(0, np.iinfo(e).max, (NB, bs, Hk, D), dtype=e)
    return kc, rng.integers(0, np.iinfo(e).max, kc.shape, dtype=e), None


def on_gpu(x, dtype):
    if x is None:
        return None
    if dtype in ("int4", "e4m3"):
        return torch.from_numpy(x).to(dev())
    signed = x.view(np.int32 if x.dtype == np.uint32 else np.int16)
    return torch.from_numpy(signed).to(dev()).view(cc.TORCH[dtype])


def back(t, like):
    if t is None:
        return None
    if t.dtype in (torch.uint8, torch.float16) and like.dtype in (np.uint8, np.float16):
        return t.cpu().numpy()
    return t.view(torch.int32 if like.dtype == np.uint32 else torch.int16).cpu().numpy().view(like.dtype)


def reference(case, mass, lens, keep, recent, bt, obt, bs, kept_len, out_len, arrays, int4):
    """Expected (kept, mass_out, arrays): rows moved from a copy of the arrays as they were."""
    B, Hk, _ = mass.shape
    kept = np.full((B, Hk, kept_len), -1, np.int32)
    mo = np.zeros((B, Hk, out_len), np.float32)
    old = [None if a is None else a.copy() for a in arrays]
    new = [None if a is None else a.copy() for a in arrays]
    for b in range(B):
        c, n = int(lens[b]), min(int(lens[b]), int(keep[b]))
        for h in range(Hk):
            at = cc.evict(mass[b, h], c, int(keep[b]), recent)
            kept[b, h, :n] = at
            mo[b, h, :n] = mass[b, h, at]
            i = np.arange(n)
            sb, so, db, do = bt[b, at // bs], at % bs, obt[b, i // bs], i % bs
            for o, a in zip(old, new):
                if a is None:
                    continue
                if int4:
                    a[db, h, do] = o[sb, h, so]
                else:
                    a[db, do, h] = o[sb, so, h]
    return kept, mo, new


def run_case(pa, seed, lens, keep, recent, Hk, D, bs, dtype, kind="plain", in_place=False, extra=5):
    rng = np.random.default_rng(seed)
    lens, keep = np.asarray(lens, np.int32), np.asarray(keep, np.int32)
    bt, nb, _ = cc.tables(rng, lens, bs)
    top = int(max(1, np.minimum(lens, keep).max()))
    if in_place:
        obt, NB = bt, nb
    else:
        obt, extra_blocks, _ = cc.tables(rng, np.minimum(lens, keep), bs)
        obt = np.where(obt >= 0, obt + nb, -1).astype(np.int32)
        NB = nb + extra_blocks
    B, M = len(lens), int(max(1, lens.max())) + extra
    mass = masses(rng, (B, Hk, M), kind)
    arrays = caches(rng, NB, bs, Hk, D, dtype)
    kept_len = top + 3
    t = [on_gpu(a, dtype if i < 2 else "int4") for i, a in enumerate(arrays)]
    md = torch.from_numpy(mass).to(dev())
    out_len = M if in_place else top + 7
    mo = md if in_place else torch.full((B, Hk, out_len), 9.0, device=dev())
    kd = torch.full((B, Hk, kept_len), 77, dtype=torch.int32, device=dev())
    btd = torch.from_numpy(bt).to(dev())
    pa.paged_kv_evict(kd, md, mo, t[0], t[1], btd, btd if in_place else torch.from_numpy(obt).to(dev()),
                      torch.from_numpy(lens).to(dev()), torch.from_numpy(keep).to(dev()), recent, kv_params=t[2])
    assert pa.get_device_error() == 0
    kept, want_mo, want = reference(None, mass, lens, keep, recent, bt, obt, bs, kept_len, out_len, arrays,
                                    dtype == "int4")
    assert np.array_equal(kd.cpu().numpy(), kept)
    assert np.array_equal(mo.cpu().numpy().view(np.uint32), want_mo.view(np.uint32))
    for got, w in zip(t, want):
        if w is not None:
            assert np.array_equal(back(got, w).view(np.uint8), w.view(np.uint8))
    if not in_place:
        assert np.array_equal(md.cpu().numpy().view(np.uint32), mass.view(np.uint32))


LENS = [1, 5, 0, 16, 17, 100, 1023, 1024, 1025, 2500, 64, 300]
KEEP = [1, 9, 4, 16, 1, 40, 1000, 1024, 512, 1100, 0, 299]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,Hk,D,bs", [("bf16", 2, 128, 16), ("f16", 1, 64, 8), ("f32", 3, 64, 4), ("e4m3", 2, 128, 16),
                                           ("int4", 2, 128, 16), ("int4", 3, 64, 8), ("bf16", 1, 96, 1),
                                           ("bf16", 2, 128, 256)])
def test_evict_is_bit_exact(pa, dtype, Hk, D, bs, in_place):
    run_case(pa, 3 + D + bs, LENS, KEEP, 7, Hk, D, bs, dtype, in_place=in_place)


@pytest.mark.parametrize("kind", ["ties", "equal", "special", "crowd"])
@pytest.mark.parametrize("recent", [0, 1, 33, 100000])
def test_evict_ties_and_special_masses(pa, kind, recent):
    for in_place in (False, True):
        run_case(pa, 17, LENS, KEEP, recent, 2, 64, 16, "bf16", kind=kind, in_place=in_place)


@pytest.mark.parametrize("keep,recent", [(8192, 512), (39999, 1), (3, 2), (40000, 0)])
def test_evict_long(pa, keep, recent):
    run_case(pa, 29, [40000, 12345], [keep, keep], recent, 1, 128, 16, "int4")
    run_case(pa, 30, [40000, 12345], [keep, keep], recent, 2, 64, 64, "bf16", kind="ties", in_place=True)
    run_case(pa, 31, [40000, 12345], [keep, keep], recent, 1, 64, 64, "f16", kind="crowd", in_place=True)


def test_evict_rows_beyond_a_cluster(pa):
    """A row too long for the selection's shared memory, next to a short one."""
    run_case(pa, 37, [430000, 700], [300, 400], 50, 1, 64, 256, "int4", extra=0)
    run_case(pa, 38, [430000, 700], [429000, 400], 50, 1, 64, 256, "int4", kind="ties", in_place=True, extra=0)


@pytest.mark.parametrize("kind", ["equal", "crowd"])
def test_evict_long_list_in_one_cta(pa, kind):
    """As many rows as give each one CTA, with more masses of the threshold's first digit than its list holds."""
    run_case(pa, 41, [2900] * 160, [1500] * 160, 9, 2, 64, 64, "int4", kind=kind, in_place=True)


@pytest.mark.parametrize("B", [1, 20, 90])
def test_evict_batch_sizes(pa, B):
    """From whole clusters for a row to one CTA."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 700, B)
    keep = np.minimum(rng.integers(0, 600, B), lens)
    run_case(pa, 39 + B, lens, keep, 11, 2, 128, 16, "bf16", kind="special", in_place=B == 20)


def test_evict_own_blocks_named_by_a_shorter_table(pa):
    """Eviction in place through another tensor that names the first blocks of each sequence."""
    rng = np.random.default_rng(33)
    lens, keep = np.array([500, 90], np.int32), np.array([100, 50], np.int32)
    bt, NB, _ = cc.tables(rng, lens, 16)
    obt = bt[:, :7].copy()
    kc, vc, _ = caches(rng, NB, 16, 2, 128, "bf16")
    mass = masses(rng, (2, 2, 500), "plain")
    kept, mo, want = reference(None, mass, lens, keep, 10, bt, obt, 16, 100, 100, (kc, vc, None), False)
    t = [on_gpu(a, "bf16") for a in (kc, vc)]
    kd = torch.empty((2, 2, 100), dtype=torch.int32, device=dev())
    mod = torch.empty((2, 2, 100), device=dev())
    pa.paged_kv_evict(kd, torch.from_numpy(mass).to(dev()), mod, *t, torch.from_numpy(bt).to(dev()),
                      torch.from_numpy(obt).to(dev()), torch.from_numpy(lens).to(dev()),
                      torch.from_numpy(keep).to(dev()), 10)
    assert np.array_equal(kd.cpu().numpy(), kept) and np.array_equal(mod.cpu().numpy(), mo)
    assert np.array_equal(back(t[0], kc), want[0]) and np.array_equal(back(t[1], vc), want[1])


def test_evict_device_errors(pa):
    """Lengths out of range are cut, rows of bad blocks stay; both are reported."""
    d = dev()
    rng = np.random.default_rng(35)
    kc, vc, _ = caches(rng, 12, 16, 1, 64, "bf16")
    bt = np.arange(12, dtype=np.int32).reshape(3, 4)
    mass = masses(rng, (3, 1, 64), "plain")

    def call(lens, keep, table=bt, out=bt, kept_len=64, mo_len=64):
        t = [on_gpu(a, "bf16") for a in (kc, vc)]
        kd = torch.full((3, 1, kept_len), 5, dtype=torch.int32, device=d)
        mo = torch.empty((3, 1, mo_len), device=d)
        pa.paged_kv_evict(kd, torch.from_numpy(mass).to(d), mo, *t, torch.from_numpy(table).to(d),
                          torch.from_numpy(out).to(d), torch.tensor(lens, dtype=torch.int32, device=d),
                          torch.tensor(keep, dtype=torch.int32, device=d), 2)
        return kd.cpu().numpy(), back(t[0], kc)

    kd, _ = call([64, -4, 64], [20, 20, 20])
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT
    assert (kd[1] == -1).all() and (kd[0, 0, :20] >= 0).all()
    kd, _ = call([64, 65, 64], [20, 20, -1])
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT
    assert (kd[2] == -1).all() and np.array_equal(kd[1, 0, :20], cc.evict(mass[1, 0], 64, 20, 2))
    kd, _ = call([64, 64, 64], [20, 20, 30], kept_len=20)
    assert pa.get_device_error() == pa.PA_DEVERR_CONTEXT
    assert np.array_equal(kd[2, 0, :20], cc.evict(mass[2, 0], 64, 20, 2))
    bad = bt.copy()
    bad[1, 1] = 400
    bad[2, 0] = -1
    _, got = call([64, 64, 64], [20, 20, 20], table=bad)
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
    _, got = call([64, 64, 64], [20, 20, 20], out=bad)
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(got[8:], kc[8:9].repeat(4, 0)) or np.array_equal(got[8], kc[8])


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("int4", [False, True])
def test_serving_run(pa, int4):
    """A prompt is written, decoded for some steps that accumulate weights, cut back in place, and
    decoded on; every step is checked against the formula over the tokens that are left. The
    4-bit cache is also read back into a 16-bit one, whose prefill must agree with its decode."""
    rng = np.random.default_rng(90)
    d = dev()
    B, H, Hk, D, bs, steps, keep, recent = 3, 16, 4, 128, 16, 5, 60, 9
    prompt = np.array([130, 47, 64])
    M = int(prompt.max()) + 2 * steps
    bt, NB, _ = cc.tables(rng, prompt + 2 * steps, bs)
    btd = torch.from_numpy(bt).to(d)
    if int4:
        kc = torch.zeros((NB, Hk, bs, D // 2), dtype=torch.uint8, device=d)
        vc = torch.zeros_like(kc)
        par = torch.full((NB, Hk, bs, 4), float("nan"), dtype=torch.float16, device=d)
    else:
        kc = torch.full((NB, bs, Hk, D), float("nan"), dtype=torch.bfloat16, device=d)
        vc = torch.full_like(kc, float("nan"))
        par = None
    # per sequence and kv head: the rows that are left, as held by the cache
    held = [[([], []) for _ in range(Hk)] for _ in range(B)]

    def put(b, pos, x_k, x_v):
        slots = torch.from_numpy((bt[b, pos // bs].astype(np.int64) * bs + pos % bs).astype(np.int32)).to(d)
        k, v = (torch.from_numpy(x).to(d).bfloat16() for x in (x_k, x_v))
        if int4:
            pa.paged_kv_write_int4(k, v, slots, kc, vc, par)
        else:
            pa.paged_kv_write(k, v, slots, kc, vc)
        for x, i in ((x_k, 0), (x_v, 1)):
            val = cc.stored(x, "bf16")
            if int4:
                val = cc.values(*cc.cache_rows(val.astype(np.float32)))
            for h in range(Hk):
                held[b][h][i].extend(val[:, h])

    lens = prompt.copy()
    for b in range(B):
        put(b, np.arange(prompt[b]), rng.standard_normal((prompt[b], Hk, D)).astype(np.float32),
            rng.standard_normal((prompt[b], Hk, D)).astype(np.float32))
    mass = torch.zeros((B, Hk, M), device=d)
    ref_mass = np.zeros((B, Hk, M))

    def step():
        for b in range(B):
            put(b, np.array([lens[b]]), rng.standard_normal((1, Hk, D)).astype(np.float32),
                rng.standard_normal((1, Hk, D)).astype(np.float32))
            lens[b] += 1
        q = rng.standard_normal((B, H, D)).astype(np.float32) * np.float32(2.0)
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=d)
        cl = torch.tensor(lens, dtype=torch.int32, device=d)
        qd = torch.from_numpy(q).to(d).bfloat16()
        if int4:
            pa.paged_attention_decode_int4(out, qd, kc, vc, par, btd, cl, D ** -0.5, mass=mass)
        else:
            pa.paged_attention_decode_scored(out, qd, mass, kc, vc, btd, cl, D ** -0.5)
        got = out.double().cpu().numpy()
        qs = cc.stored(q, "bf16")
        for b in range(B):
            for h in range(Hk):
                k, v = (np.asarray(held[b][h][i])[:, None] for i in (0, 1))
                ref, w, big, wv = cc.attention(qs[b, 4 * h:4 * h + 4], k, v, D ** -0.5)
                # output rounding, the 16-bit weights (bf16 at most: 2^-8), the scores' errors
                dx = 3 * big.max() * (D + 2) * 2.0 ** -23
                tol = np.abs(ref) * 2.0 ** -8 + (2.0 ** -8 + 4 * np.expm1(2 * dx) + 2.0 ** -10) * wv
                assert (np.abs(got[b, 4 * h:4 * h + 4] - ref) <= tol).all()
                ref_mass[b, h, :lens[b]] += w.sum(0)
        return qd, out

    for _ in range(steps):
        step()
    m = mass.cpu().numpy()
    assert np.abs(m - ref_mass).max() <= 1e-3 * max(1.0, ref_mass.max())   # scores off by dx < 1e-4 a step
    kept = torch.empty((B, Hk, keep), dtype=torch.int32, device=d)
    pa.paged_kv_evict(kept, mass, mass, kc, vc, btd, btd, torch.tensor(lens, dtype=torch.int32, device=d),
                      torch.full((B,), keep, dtype=torch.int32, device=d), recent, kv_params=par)
    for b in range(B):
        n = min(int(lens[b]), keep)
        for h in range(Hk):
            at = cc.evict(m[b, h], int(lens[b]), keep, recent)
            assert np.array_equal(kept[b, h, :n].cpu().numpy(), at)
            held[b][h] = tuple([held[b][h][i][j] for j in at] for i in (0, 1))
            ref_mass[b, h] = 0.0
            ref_mass[b, h, :n] = m[b, h, at]
        lens[b] = n
    assert np.array_equal(mass.cpu().numpy(), ref_mass.astype(np.float32))
    for _ in range(steps):
        qd, out = step()
    if int4:
        # read back, and attended by the prefill kernel with one-token chunks
        n16 = [-(-int(x) // bs) for x in lens]
        bt16 = torch.full((B, max(n16)), -1, dtype=torch.int32, device=d)
        slots = []
        for b in range(B):
            bt16[b, :n16[b]] = torch.arange(sum(n16[:b]), sum(n16[:b + 1]), dtype=torch.int32, device=d)
            s = np.full(n16[b] * bs, -1, np.int32)
            s[:lens[b]] = cc.slots_of(bt[b], lens[b], bs)
            slots.append(s)
        k16 = torch.zeros((sum(n16), bs, Hk, D), dtype=torch.bfloat16, device=d)
        v16 = torch.zeros_like(k16)
        pa.paged_kv_read_int4(k16.view(-1, Hk, D), v16.view(-1, Hk, D), torch.from_numpy(np.concatenate(slots)).to(d),
                              kc, vc, par)
        pre = torch.empty_like(out)
        pa.paged_attention_prefill(pre, qd, k16, v16, bt16, torch.tensor(lens, dtype=torch.int32, device=d),
                                   torch.arange(B + 1, dtype=torch.int32, device=d), D ** -0.5, 1)
        # K and V rounded to bf16 on the way: scores off by 2^-9 of |q||k| scale (about 0.03), weights alike
        assert (pre.float() - out.float()).abs().max() < 0.15
    assert pa.get_device_error() == 0
