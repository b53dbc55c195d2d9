"""Host side of the cache-compression calls (no GPU): what is refused before any CUDA call,
the sizes of their workspaces, and pins of the plain forms the GPU tests compare with."""
import numpy as np
import pytest

import compress_cases as cc


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build
    build()
    import paged_kv_cache_261_gb300 as pa
    return pa


INVALID, UNSUPPORTED = -1, -2


def _rw(pa, name, **kw):
    a = dict(k=16, v=16, slots=16, T=4, kc=16, vc=16, par=16, nb=8, bs=16, Hk=2, D=128, dt=2)
    a.update(kw)
    order = ("k", "v", "slots", "T", "kc", "vc", "par", "nb", "bs", "Hk", "D", "dt")
    return getattr(pa.lib(), name)(*[a[x] for x in order], None)


@pytest.mark.parametrize("name", ["pa_paged_kv_write_int4", "pa_paged_kv_read_int4"])
@pytest.mark.parametrize("bad,code", [
    (dict(D=96), UNSUPPORTED), (dict(D=0), INVALID), (dict(bs=12), UNSUPPORTED), (dict(bs=4), UNSUPPORTED),
    (dict(bs=512), UNSUPPORTED), (dict(Hk=0), INVALID), (dict(nb=0), INVALID), (dict(T=-1), INVALID),
    (dict(dt=3), INVALID), (dict(dt=4), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(slots=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(par=None), INVALID),
    (dict(k=8), INVALID), (dict(kc=8), INVALID), (dict(par=8), INVALID), (dict(nb=1 << 62), INVALID),
    (dict(T=0), 0), (dict(T=1 << 60), UNSUPPORTED)])
def test_int4_rows_refusals(pa, name, bad, code):
    assert _rw(pa, name, **bad) == code


def test_copy_blocks_int4_refusals(pa):
    def call(kc=16, vc=16, par=16, pairs=16, n=1, nb=8, bs=16, Hk=2, D=128):
        return pa.lib().pa_copy_blocks_int4(kc, vc, par, pairs, n, nb, bs, Hk, D, None)
    assert call(D=80) == UNSUPPORTED and call(bs=24) == UNSUPPORTED and call(n=-1) == INVALID
    assert call(par=None) == INVALID and call(par=8) == INVALID and call(pairs=None) == INVALID
    assert call(n=0) == 0


def _decode(pa, **kw):
    a = dict(out=16, q=16, kc=16, vc=16, par=16, mass=None, ml=0, bt=16, mb=4, cl=16, B=2, H=8, Hk=2, D=128, bs=16,
             nb=64, scale=0.1, mc=0, ws=None, wsb=0, dt=2)
    a.update(kw)
    order = ("out", "q", "kc", "vc", "par", "mass", "ml", "bt", "mb", "cl", "B", "H", "Hk", "D", "bs", "nb", "scale",
             "mc", "ws", "wsb", "dt")
    return pa.lib().pa_paged_attention_decode_int4(*[a[x] for x in order], None)


@pytest.mark.parametrize("bad,code", [
    (dict(H=6, Hk=4), INVALID), (dict(D=96), UNSUPPORTED), (dict(bs=12), UNSUPPORTED), (dict(bs=4), UNSUPPORTED),
    (dict(bs=512), UNSUPPORTED), (dict(H=64, Hk=2), UNSUPPORTED), (dict(dt=0), UNSUPPORTED), (dict(dt=3), INVALID), (dict(dt=9), INVALID), (dict(out=None), INVALID),
    (dict(par=None), INVALID), (dict(par=8), INVALID), (dict(q=8), INVALID), (dict(nb=0), INVALID),
    (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(mc=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(mass=16, ml=0), INVALID), (dict(mass=18, ml=9), INVALID), (dict(B=0), 0)])
def test_decode_int4_refusals(pa, bad, code):
    assert _decode(pa, **bad) == code


def _scored(pa, **kw):
    a = dict(out=16, q=16, mass=16, ml=64, kc=16, vc=16, bt=16, mb=4, cl=16, B=2, H=8, Hk=2, D=128, bs=16,
             nb=64, scale=0.1, mc=0, part=0, ws=None, wsb=0, dt=2)
    a.update(kw)
    order = ("out", "q", "mass", "ml", "kc", "vc", "bt", "mb", "cl", "B", "H", "Hk", "D", "bs", "nb", "scale",
             "mc", "part", "ws", "wsb", "dt")
    return pa.lib().pa_paged_attention_decode_scored(*[a[x] for x in order], None)


@pytest.mark.parametrize("bad,code", [
    (dict(H=6, Hk=4), INVALID), (dict(D=96), UNSUPPORTED), (dict(bs=12), UNSUPPORTED), (dict(H=64, Hk=2), UNSUPPORTED),
    (dict(part=100), INVALID), (dict(dt=3), INVALID), (dict(mass=None), INVALID), (dict(ml=0), INVALID),
    (dict(mass=2), INVALID), (dict(kc=8), INVALID), (dict(cl=None), INVALID), (dict(B=0), 0)])
def test_decode_scored_refusals(pa, bad, code):
    assert _scored(pa, **bad) == code


def _evict(pa, **kw):
    a = dict(kept=16, kl=8, mass=16, ml=64, mo=16, mol=8, kc=16, vc=16, par=None, bt=16, mb=4, obt=16, omb=1, cl=16,
             kp=16, recent=2, B=2, Hk=2, D=128, bs=16, nb=64, dt=2)
    a.update(kw)
    order = ("kept", "kl", "mass", "ml", "mo", "mol", "kc", "vc", "par", "bt", "mb", "obt", "omb", "cl", "kp", "recent",
             "B", "Hk", "D", "bs", "nb", "dt")
    return pa.lib().pa_paged_kv_evict(*[a[x] for x in order], None)


@pytest.mark.parametrize("bad,code", [
    (dict(recent=-1), INVALID), (dict(kl=0), INVALID), (dict(ml=0), INVALID), (dict(mol=0), INVALID),
    (dict(mb=0), INVALID), (dict(omb=0), INVALID), (dict(dt=5), INVALID), (dict(dt=-1), INVALID),
    (dict(D=100), UNSUPPORTED), (dict(D=8200), UNSUPPORTED), (dict(bs=12), UNSUPPORTED), (dict(bs=512), UNSUPPORTED), (dict(B=70000), UNSUPPORTED),
    (dict(kept=None), INVALID), (dict(mass=None), INVALID), (dict(mo=None), INVALID), (dict(obt=None), INVALID),
    (dict(kp=None), INVALID), (dict(kc=8), INVALID), (dict(mass=2), INVALID), (dict(kept=2), INVALID),
    (dict(dt=4), INVALID), (dict(dt=4, par=8), INVALID), (dict(dt=4, par=16, D=96), UNSUPPORTED),
    (dict(dt=4, par=16, bs=4), UNSUPPORTED), (dict(nb=1 << 62), INVALID), (dict(B=0), 0)])
def test_evict_refusals(pa, bad, code):
    assert _evict(pa, **bad) == code


def test_evict_refuses_overlapping_masses(pa):
    # rows of 64 masses, 2 sequences of 2 kv heads: 1024 bytes from 4096 on; 8 a row out: 128 bytes
    for mo, mol in ((4096, 8), (4100, 64), (3972, 8), (5116, 8), (4096, 65)):
        assert _evict(pa, mass=4096, mo=mo, mol=mol) == INVALID
    assert _evict(pa, mass=4096, ml=1 << 62, mo=1 << 20) == INVALID


def test_contexts_past_the_token_count_are_refused(pa):
    top = 2 ** 31 - 1
    assert _decode(pa, mc=top) == UNSUPPORTED and _decode(pa, mb=2 ** 31 // 16, mc=0) == UNSUPPORTED
    assert _scored(pa, mc=top) == UNSUPPORTED


def test_python_checks_refuse_host_tensors_and_wrong_shapes(pa):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 2, 128)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    p = torch.zeros(4, 2, 16, 4, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: pa.paged_kv_write_int4(x, x, i, c, c, p), lambda: pa.paged_kv_read_int4(x, x, i, c, c, p),
                 lambda: pa.paged_attention_decode_int4(x, x, c, c, p, i, i, 1.0),
                 lambda: pa.paged_attention_decode_scored(x, x, x, x, x, i, i, 1.0),
                 lambda: pa.paged_kv_evict(i, x, x, x, x, i, i, i, i, 0), lambda: pa.copy_blocks(c, c, i, kv_params=p)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


def test_workspace_sizes(pa):
    for B, H, Hk, D, ctx, part in ((1, 8, 8, 128, 700, 0), (64, 32, 8, 128, 4096, 0), (8, 64, 8, 64, 131072, 512),
                                   (4000, 12, 1, 64, 50, 0)):
        # a partial of a group for every warp of the grid and every row, with and without the scores
        n, with_mass = (pa.decode_int4_workspace_bytes(B, H, Hk, D, ctx, w) for w in (False, True))
        assert n >= min(B, 1536) * Hk * (8 + H // Hk * (8 + 4 * D))
        # the scores: the heads of a group rounded up to 2, 4, 8 or 16, the tokens to a multiple of 4
        G = H // Hk
        scores = B * Hk * (2 if G <= 2 else 4 if G <= 4 else 8 if G <= 8 else 16) * -(-ctx // 4) * 16
        assert 0 <= with_mass - n - B * H * 8 - scores < 256
        P = -(-ctx // pa.decode_partition_size(B, ctx, part))
        split = B * H * P * (2 + D) * 4 if P > 1 else 0
        n = pa.decode_scored_workspace_bytes(B, H, Hk, D, ctx, part)
        assert 0 <= n - (split + B * H * P * 8 + scores) < 3 * 256
    # a larger batch never needs less
    sizes = [pa.decode_int4_workspace_bytes(B, 32, 8, 128, 2048) for B in (1, 2, 64, 512, 5000)]
    assert sizes == sorted(sizes)
    assert pa.decode_int4_workspace_bytes(0, 8, 2, 128, 100) == 0
    assert pa.decode_int4_workspace_bytes(2, 9, 2, 128, 100) == 0


def test_plain_quantisation_pins():
    # range 0..15 with step 1: codes are the values; halves go to the even code
    x = np.arange(16, dtype=np.float32)
    n, s, z = cc.quantise(np.concatenate([x, x + np.float32(0.5)]).clip(0, 15)[None])
    assert s[0] == 1.0 and z[0] == 0.0
    assert n[0, :16].tolist() == list(range(16))
    assert n[0, 16:].tolist() == [0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14, 15]
    b = cc.pack(n)
    assert b[0, 1] == 0x32 and np.array_equal(cc.unpack(b), n)
    assert np.array_equal(cc.values(b, s, z), n.astype(np.float64))
    n, s, z = cc.quantise(np.full((1, 64), 2.5, np.float32))
    assert s[0] == 0 and z[0] == 2.5 and not n.any()
    n, s, z = cc.quantise(np.array([[1.0, np.nan] * 32], np.float32))
    assert np.isnan(s[0]) and np.isnan(z[0]) and not n.any()


def test_plain_eviction_pins():
    m = np.array([3.0, 1.0, 3.0, 2.0, 9.0, 9.0], np.float32)
    assert cc.evict(m, 6, 3, 0).tolist() == [0, 4, 5]          # 3.0 twice: the lower index
    assert cc.evict(m, 6, 3, 1).tolist() == [0, 4, 5]
    assert cc.evict(m, 4, 3, 1).tolist() == [0, 2, 3]
    assert cc.evict(m, 4, 2, 5).tolist() == [2, 3]
    assert cc.evict(m, 2, 9, 1).tolist() == [0, 1]
    assert cc.evict(np.array([np.nan, -np.inf, np.nan, 0.0], np.float32), 4, 2, 0).tolist() == [1, 3]
    assert cc.evict(np.array([np.nan, -0.0, 0.0], np.float32), 3, 2, 0).tolist() == [1, 2]
