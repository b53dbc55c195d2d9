"""Host side of a serving step's calls (no GPU): what is refused before any CUDA call, workspace
sizes, the rotary frequencies, and pins of the plain forms the GPU tests compare with."""
import numpy as np
import pytest

import step_cases as sc


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build
    build()
    import paged_kv_cache_261_gb300 as pa
    return pa


INVALID, UNSUPPORTED = -1, -2


def _append(pa, **kw):
    a = dict(bt=16, mb=4, cl=16, ncl=16, ql=16, B=2, free=16, cap=8, nf=16, nnf=16, start=16, slots=16, pos=16, T=4,
             bs=16, nb=8)
    a.update(kw)
    return pa.lib().pa_paged_blocks_append(*a.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(mb=0), INVALID), (dict(B=-1), INVALID), (dict(B=16385), UNSUPPORTED), (dict(cap=-1), INVALID),
    (dict(cap=1 << 31), UNSUPPORTED), (dict(bs=0), INVALID), (dict(bs=12), UNSUPPORTED), (dict(bs=512), UNSUPPORTED),
    (dict(nb=0), INVALID), (dict(nb=1 << 27), UNSUPPORTED), (dict(T=-1), INVALID), (dict(T=2 ** 31 - 1), UNSUPPORTED),
    (dict(T=2 ** 30 + 1), UNSUPPORTED), (dict(cap=2 ** 30 + 1), UNSUPPORTED), (dict(bt=None), INVALID), (dict(cl=None), INVALID), (dict(ncl=None), INVALID), (dict(ql=None), INVALID),
    (dict(free=None), INVALID), (dict(nf=None), INVALID), (dict(nnf=None), INVALID), (dict(start=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID)])
def test_append_refusals(pa, bad, code):
    assert _append(pa, **bad) == code


def _release(pa, **kw):
    a = dict(bt=16, mb=4, cl=16, ncl=16, fin=16, B=2, free=16, cap=8, nf=16, nnf=16, bs=16, nb=8)
    a.update(kw)
    return pa.lib().pa_paged_blocks_release(*a.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(mb=0), INVALID), (dict(B=-1), INVALID), (dict(B=16385), UNSUPPORTED), (dict(cap=-1), INVALID),
    (dict(bs=24), UNSUPPORTED), (dict(nb=0), INVALID), (dict(nb=1 << 27), UNSUPPORTED), (dict(bt=None), INVALID),
    (dict(cl=None), INVALID), (dict(ncl=None), INVALID), (dict(fin=None), INVALID), (dict(free=None), INVALID),
    (dict(nf=None), INVALID), (dict(nnf=None), INVALID)])
def test_release_refusals(pa, bad, code):
    assert _release(pa, **bad) == code


def _rotary(pa, **kw):
    a = dict(qo=16, qos=512, ko=16, kos=256, q=16, qs=512, k=16, ks=256, pos=16, f=16, factor=1.0, inter=0, T=4, H=4,
             Hk=2, D=128, rd=128, dt=2)
    a.update(kw)
    return pa.lib().pa_rotary_embedding(*a.values(), None)


ROTARY_BAD = [
    (dict(T=-1), INVALID), (dict(T=0), 0), (dict(T=1 << 31), UNSUPPORTED), (dict(H=0), INVALID),
    (dict(D=0), INVALID), (dict(D=136), UNSUPPORTED), (dict(D=2048, qs=8192, qos=8192), UNSUPPORTED),
    (dict(rd=0), INVALID), (dict(rd=144), INVALID), (dict(rd=24), UNSUPPORTED), (dict(dt=3), INVALID),
    (dict(dt=9), INVALID), (dict(factor=float("nan")), INVALID), (dict(q=None), INVALID), (dict(q=8), INVALID),
    (dict(qo=None), INVALID), (dict(qo=8), INVALID), (dict(k=None), INVALID), (dict(pos=None), INVALID),
    (dict(f=None), INVALID), (dict(f=4), INVALID), (dict(qs=-512), INVALID), (dict(qs=516), INVALID),
    (dict(qos=504), INVALID), (dict(qos=0), INVALID), (dict(ks=4), INVALID), (dict(qs=1 << 62), INVALID)]


@pytest.mark.parametrize("bad,code", ROTARY_BAD + [
    (dict(Hk=-1), INVALID), (dict(ko=None), INVALID), (dict(ko=8), INVALID), (dict(kos=248), INVALID)])
def test_rotary_refusals(pa, bad, code):
    assert _rotary(pa, **bad) == code


def _write_rotary(pa, **kw):
    a = dict(qo=16, qos=512, q=16, qs=512, k=16, ks=256, v=16, vs=256, pos=16, f=16, factor=1.0, inter=0, slots=16, T=4,
             kc=16, vc=16, nb=8, bs=16, H=4, Hk=2, D=128, rd=128, dt=2)
    a.update(kw)
    return pa.lib().pa_paged_kv_write_rotary(*a.values(), None)


@pytest.mark.parametrize("bad,code", ROTARY_BAD + [
    (dict(Hk=0), INVALID), (dict(nb=0), INVALID), (dict(nb=1 << 62), INVALID), (dict(bs=0), INVALID),
    (dict(v=None), INVALID), (dict(v=8), INVALID), (dict(vs=12), INVALID), (dict(slots=None), INVALID),
    (dict(kc=None), INVALID), (dict(kc=8), INVALID), (dict(vc=None), INVALID)])
def test_write_rotary_refusals(pa, bad, code):
    assert _write_rotary(pa, **bad) == code


def _block_rw(pa, write, **kw):
    a = dict(k=16, ks=256, v=16, vs=256, slots=16, T=4, kc=16, vc=16, sc=16, nb=8, bs=16, Hk=2, D=128, dt=2)
    a.update(kw)
    if not write:
        del a["ks"], a["vs"]
    return getattr(pa.lib(), f"pa_paged_kv_{'write' if write else 'read'}_fp8_block")(*a.values(), None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("bad,code", [
    (dict(D=96), UNSUPPORTED), (dict(D=0), INVALID), (dict(bs=12), UNSUPPORTED), (dict(bs=4), UNSUPPORTED),
    (dict(bs=512), UNSUPPORTED), (dict(Hk=0), INVALID), (dict(nb=0), INVALID), (dict(T=-1), INVALID),
    (dict(dt=3), INVALID), (dict(dt=4), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(slots=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(sc=None), INVALID),
    (dict(k=8), INVALID), (dict(kc=8), INVALID), (dict(sc=8), INVALID), (dict(nb=1 << 62), INVALID),
    (dict(T=0), 0), (dict(T=1 << 60), UNSUPPORTED)])
def test_block_scaled_rows_refusals(pa, write, bad, code):
    assert _block_rw(pa, write, **bad) == code


@pytest.mark.parametrize("bad", [dict(ks=-256), dict(ks=260), dict(vs=4), dict(vs=1 << 62)])
def test_block_scaled_write_refuses_strides(pa, bad):
    assert _block_rw(pa, True, **bad) == INVALID


def test_copy_blocks_fp8_block_refusals(pa):
    def call(kc=16, vc=16, sc=16, pairs=16, n=1, nb=8, bs=16, Hk=2, D=128):
        return pa.lib().pa_copy_blocks_fp8_block(kc, vc, sc, pairs, n, nb, bs, Hk, D, None)
    assert call(D=80) == UNSUPPORTED and call(bs=24) == UNSUPPORTED and call(n=-1) == INVALID
    assert call(sc=None) == INVALID and call(sc=8) == INVALID and call(pairs=None) == INVALID
    assert call(Hk=70000) == UNSUPPORTED and call(n=1 << 31) == UNSUPPORTED and call(n=0) == 0


def _decode(pa, **kw):
    a = dict(out=16, q=16, kc=16, vc=16, sc=16, bt=16, mb=4, cl=16, B=2, H=8, Hk=2, D=128, bs=16, nb=64, scale=0.1,
             mc=0, ws=None, wsb=0, dt=2)
    a.update(kw)
    return pa.lib().pa_paged_attention_decode_fp8_block(*a.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(H=6, Hk=4), INVALID), (dict(D=96), UNSUPPORTED), (dict(bs=12), UNSUPPORTED), (dict(bs=4), UNSUPPORTED),
    (dict(bs=512), UNSUPPORTED), (dict(H=64, Hk=2), UNSUPPORTED), (dict(dt=0), UNSUPPORTED), (dict(dt=3), INVALID),
    (dict(out=None), INVALID), (dict(sc=None), INVALID), (dict(sc=8), INVALID), (dict(q=8), INVALID),
    (dict(nb=0), INVALID), (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(mc=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(mc=2 ** 31 - 1), UNSUPPORTED), (dict(mb=2 ** 31 // 16), UNSUPPORTED),
    (dict(B=0), 0)])
def test_decode_fp8_block_refusals(pa, bad, code):
    assert _decode(pa, **bad) == code


def test_python_checks_refuse_host_tensors_and_wrong_shapes(pa):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 2, 128)
    c = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    s = torch.zeros(4, 2, 2)
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(64, dtype=torch.float64)
    for call in (lambda: pa.paged_kv_write_fp8_block(x, x, i, c, c, s), lambda: pa.paged_kv_read_fp8_block(x, x, i, c, c, s),
                 lambda: pa.paged_attention_decode_fp8_block(x, x, c, c, s, i, i, 1.0),
                 lambda: pa.copy_blocks(c, c, i, kv_scales=s), lambda: pa.rotary_embedding(x, x, x, x, i, f),
                 lambda: pa.paged_kv_write_rotary(x, x, x, x, i, f, i, x, x),
                 lambda: pa.paged_blocks_append(i, i, i, i, i, i, i, i, 16, 8),
                 lambda: pa.paged_blocks_release(i, i, i.bool(), i, i, 16)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="kv_params belongs"):
        pa.copy_blocks(c, c, i, kv_params=s, kv_scales=s)


def test_workspace_sizes(pa):
    for B, H, Hk, D, ctx in ((1, 8, 8, 128, 700), (64, 32, 8, 128, 4096), (8, 64, 8, 64, 131072), (4000, 12, 1, 64, 50)):
        n = pa.decode_fp8_block_workspace_bytes(B, H, Hk, D, ctx)
        # a row's entry, and a partial of a group for every row at least
        assert n >= min(B, 1536) * Hk * (8 + H // Hk * (8 + 4 * D))
    sizes = [pa.decode_fp8_block_workspace_bytes(B, 32, 8, 128, 2048) for B in (1, 2, 64, 512, 5000)]
    assert sizes == sorted(sizes)
    for bad in ((0, 8, 2, 128, 100), (2, 9, 2, 128, 100), (2, 8, 2, 96, 100), (2, 64, 2, 128, 100), (2, 8, 2, 128, -1)):
        assert pa.decode_fp8_block_workspace_bytes(*bad) == 0


# ---------------------------------------------------------------------------- rotary frequencies

def test_rotary_frequencies(pa):
    f = pa.rotary_frequencies(128)
    assert f.dtype == np.float64 and f.shape == (64,) and f[0] == 1.0
    assert np.allclose(f, 10000.0 ** (-np.arange(64) / 64), rtol=1e-14)
    assert np.allclose(pa.rotary_frequencies(64, 5e5, "linear", 4.0), 5e5 ** (-np.arange(32) / 32) / 4, rtol=1e-14)
    ntk = pa.rotary_frequencies(64, scaling="ntk", scale=8.0)
    plain = pa.rotary_frequencies(64)
    assert ntk[0] == plain[0] and np.isclose(ntk[-1], plain[-1] / 8, rtol=1e-12)
    for kind, kw in (("by_turns", {}), ("by_index", dict(high=32.0))):
        g = pa.rotary_frequencies(128, scaling=kind, scale=16.0, original_len=4096, **kw)
        p = pa.rotary_frequencies(128)
        ratio = p / g
        assert np.all(np.diff(ratio) >= -1e-12) and np.isclose(ratio[0], 1.0) and np.isclose(ratio[-1], 16.0)
    turns = 4096 * p / (2 * np.pi)
    g = pa.rotary_frequencies(128, scaling="by_turns", scale=16.0, original_len=4096, low=2.0, high=8.0)
    assert np.allclose(g[turns >= 8], p[turns >= 8], rtol=1e-14) and np.allclose(g[turns <= 2], p[turns <= 2] / 16, rtol=1e-14)
    mid = (turns > 2) & (turns < 8)
    k = (turns[mid] - 2) / 6
    assert mid.any() and np.allclose(g[mid], p[mid] / 16 * (1 - k) + p[mid] * k, rtol=1e-13)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, scale=0.0),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="by_turns", low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            pa.rotary_frequencies(**bad)


# ---------------------------------------------------------------------------- pins of the plain forms

def test_plain_e4m3_pins():
    assert sc.E4M3[0x08] == 2.0 ** -6 and sc.E4M3[0x01] == 2.0 ** -9 and sc.E4M3[0x7E] == 448 and sc.E4M3[0xB8] == -1.0
    codes = np.array([c for c in range(256) if c & 127 != 127 and c != 128], np.uint8)
    assert np.array_equal(sc.encode(sc.E4M3[codes]), codes)
    # ties go to the even code; beyond the largest, and infinities, to it
    x = [1 + 1 / 16, 1 + 3 / 16, 2.0 ** -10, 3 * 2.0 ** -10, 464.0, 1e9, -np.inf, -0.0, np.nan]
    assert sc.encode(x).tolist() == [0x38, 0x3A, 0x00, 0x02, 0x7E, 0x7E, 0xFE, 0x80, 0x7F]
    assert sc.scale_for(0.0) == 2.0 ** -100 and sc.scale_for(448.0) == 1.0
    assert sc.scale_for(np.nextafter(448.0, 500)) == 2.0 and sc.scale_for(224.0) == 0.5


def test_plain_scatter_pins():
    kc = np.zeros((2, 1, 8, 64), np.uint8)
    vc, s = kc.copy(), np.zeros((2, 1, 2), np.float32)
    one = np.ones((1, 1, 64))
    sc.write_blocks(kc, vc, s, 448 * one, one, [8])
    assert s[1, 0].tolist() == [1.0, 2.0 ** -8] and kc[1, 0, 0, 0] == 0x7E and vc[1, 0, 0, 0] == 0x78
    sc.write_blocks(kc, vc, s, 1792 * one, one, [9])                 # K's scale grows by 4, the older codes with it
    assert s[1, 0].tolist() == [4.0, 2.0 ** -8]
    assert kc[1, 0, 0, 0] == 0x6E and kc[1, 0, 1, 0] == 0x7E and sc.E4M3[0x6E] * 4 == 448
    sc.write_blocks(kc, vc, s, one, one, [8])                        # the first slot starts the block anew
    assert s[1, 0].tolist() == [2.0 ** -8, 2.0 ** -8] and (s[0] == 0).all()


def test_plain_layout_pins():
    table = np.array([[5, -1], [-1, -1], [7, -1]], np.int32)
    free = np.array([0, 1, 2, 3], np.int32)
    out = sc.append(table, np.array([3, 0, 4], np.int32), np.array([1, 5, 1], np.int32), free, 4, 8, 4, 8)
    assert out[0].tolist() == [[5, -1], [3, 2], [7, 1]] and out[1].tolist() == [4, 5, 5] and out[2] == 1
    assert out[3].tolist() == [0, 1, 6, 7] and out[4].tolist() == [23, 12, 13, 14, 15, 8, 4, -1]
    assert out[5].tolist() == [3, 0, 1, 2, 3, 4, 4, 0] and not out[6]
    out = sc.append(table, np.array([3, 0, 4], np.int32), np.array([1, 5, 1], np.int32), free, 1, 8, 4, 8)
    assert out[1].tolist() == [4, 0, 4] and out[2] == 1 and out[4].tolist() == [23] + [-1] * 7 and out[6] == {"free"}
    lens, f, n, err = sc.release(table, np.array([3, 0, 4], np.int32), [True, True, True], np.zeros(4, np.int32), 1, 4, 8)
    assert lens.tolist() == [0, 0, 0] and f.tolist() == [0, 5, 7, 0] and n == 3 and not err


def test_plain_rotary_pins():
    x = np.arange(8.0).reshape(1, 1, 8)
    y = sc.rotate(x, [1], np.array([np.pi / 2, 0.0]))
    assert np.allclose(y[0, 0], [-2, 1, 0, 3, 4, 5, 6, 7])
    y = sc.rotate(x, [2], np.array([np.pi / 4, 0.0]), 2.0, interleaved=True)
    assert np.allclose(y[0, 0], [-2, 0, 4, 6, 4, 5, 6, 7])


def test_host_allocator_serves_in_the_same_order(pa):
    """Appends one request after another, and frees, through the host allocator give the tables, slots
    and stack order that the plain forms of the GPU calls give."""
    rng = np.random.default_rng(1)
    bs, NB, B, MB = 4, 40, 6, 8
    al = pa.BlockAllocator(NB, bs)
    table, lens = np.full((B, MB), -1, np.int32), np.zeros(B, np.int32)
    free, nf = np.arange(NB, dtype=np.int32), NB
    for b in range(B):
        al.add_seq(b)
    for _ in range(6):
        new = rng.integers(0, 6, B).astype(np.int32)
        T = int(new.sum())
        got = sc.append(table, lens, new, free, nf, T, bs, NB)
        slots = [al.append(b, int(n))[0] for b, n in enumerate(new)]
        assert np.array_equal(np.concatenate(slots), got[4])
        table, lens, nf = got[0], got[1], got[2]
        done = rng.random(B) < 0.3
        lens, free, nf, _ = sc.release(table, lens, done, free, nf, bs, NB)
        for b in np.flatnonzero(done):
            al.free_seq(int(b))
            al.add_seq(int(b))
    assert al.stats().num_free == nf
