"""The cache-compression operators as a serving loop has them: captured in graphs, on two
streams at once, in caches past 4 GiB, with the host block allocator and forked sequences."""
import numpy as np
import pytest
import torch

import compress_cases as cc
from gpu_cases import dev, pa_mod
from test_gpu_int4 import Case, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def decode(pa, case, t, out, mass, **kw):
    pa.paged_attention_decode_int4(out, t["q"], t["kc"], t["vc"], t["par"], t["bt"], t["lens"], case.scale, mass=mass,
                                   **kw)


# ---------------------------------------------------------------------------- graphs

@pytest.mark.parametrize("workspace", ["none", "each", "shared"])
def test_two_graphs_replayed_in_turn(pa, workspace):
    """A step (write, decode with weights, eviction into other blocks, read-back) captured twice, for two
    batches of unlike sizes; the graphs are replayed in turn, with new inputs written in place, and the
    first is destroyed before the second runs on. workspace: the binding's, one of each batch's own,
    or one that both graphs hold."""
    rng = np.random.default_rng(3)
    d = dev()

    def make(seed, lens, H, Hk):
        case = Case(np.random.default_rng(seed), lens, H, Hk, 128, 16, "bf16")
        B, keep = len(lens), 40
        extra = B * -(-keep // 16)
        t = dict(case.t)
        for k in ("kc", "vc", "par"):            # room for the evicted sequences
            t[k] = torch.cat((t[k], torch.zeros((extra, *t[k].shape[1:]), dtype=t[k].dtype, device=d)))
        t["obt"] = (torch.arange(extra, dtype=torch.int32, device=d) + case.NB).view(B, -1)
        t["k"] = torch.from_numpy(rows(rng, (B, Hk, 128), "k")).to(d).bfloat16()
        t["v"] = torch.from_numpy(rows(rng, (B, Hk, 128))).to(d).bfloat16()
        t["slots"] = torch.tensor([int(case.bt[b, (n - 1) // 16]) * 16 + (n - 1) % 16 for b, n in enumerate(lens)],
                                  dtype=torch.int32, device=d)
        t["keep"] = torch.full((B,), keep, dtype=torch.int32, device=d)
        t["mass"] = torch.zeros((B, Hk, max(lens)), device=d)
        t["kept"] = torch.empty((B, Hk, keep), dtype=torch.int32, device=d)
        t["mass_out"] = torch.empty((B, Hk, keep), device=d)
        t["out"] = torch.empty_like(t["q"])
        t["ko"] = torch.zeros((extra * 16, Hk, 128), dtype=torch.bfloat16, device=d)
        t["vo"] = torch.zeros_like(t["ko"])
        t["oslots"] = torch.arange(extra * 16, dtype=torch.int32, device=d) + case.NB * 16
        n = pa.decode_int4_workspace_bytes(B, H, Hk, 128, max(lens), True)
        t["ws"] = None if workspace == "none" else torch.empty(n, dtype=torch.uint8, device=d)
        return case, t

    def step(case, t):
        pa.paged_kv_write_int4(t["k"], t["v"], t["slots"], t["kc"], t["vc"], t["par"])
        decode(pa, case, t, t["out"], t["mass"], max_context_len=int(case.lens.max()), workspace=t["ws"])
        pa.paged_kv_evict(t["kept"], t["mass"], t["mass_out"], t["kc"], t["vc"], t["bt"], t["obt"], t["lens"],
                          t["keep"], 3, kv_params=t["par"])
        pa.paged_kv_read_int4(t["ko"], t["vo"], t["oslots"], t["kc"], t["vc"], t["par"])
        return [t[k].clone() for k in ("out", "mass", "kept", "mass_out", "ko", "vo")]

    sets = [make(1, [300, 41, 77], 8, 2), make(2, [90, 2000, 40, 64, 700], 16, 4)]
    if workspace == "shared":
        sizes = [t["ws"].numel() for _, t in sets]
        for _, t in sets:
            t["ws"] = sets[sizes.index(max(sizes))][1]["ws"]
    want = []
    for case, t in sets:
        step(case, t)
        t["mass"].zero_()
        want.append(step(case, t))
        t["mass"].zero_()
    torch.cuda.synchronize()
    graphs = []
    for case, t in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(case, t)
        graphs.append(g)
    for _ in range(3):
        for (case, t), g, w in zip(sets, graphs, want):
            t["mass"].zero_()
            g.replay()
            assert all(torch.equal(t[k], x) for k, x in zip(("out", "mass", "kept", "mass_out", "ko", "vo"), w))
    graphs[0].reset()
    del graphs[0]
    torch.cuda.empty_cache()
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=d) for _ in range(8)]
    case, t = sets[1]
    t["q"].copy_((t["q"].float() * -0.5).bfloat16())
    t["mass"].zero_()
    graphs[0].replay()
    got = [t[k].clone() for k in ("out", "mass", "kept")]
    t["mass"].zero_()
    step(case, t)
    assert all(torch.equal(t[k], x) for k, x in zip(("out", "mass", "kept"), got))
    assert pa.get_device_error() == 0 and len(junk) == 8


# ---------------------------------------------------------------------------- streams

def test_two_streams_at_once(pa):
    """Back-to-back calls on two streams, each through its own cached workspace, equal the same
    calls run alone."""
    cases = [Case(np.random.default_rng(10 + i), lens, 16, 4, 128, 16, "f16")
             for i, lens in enumerate(([2500, 1, 900], [400] * 40))]
    streams = [torch.cuda.Stream() for _ in cases]
    want = []
    for c in cases:
        m = torch.zeros((len(c.lens), 4, int(c.lens.max())), device=dev())
        out = torch.empty_like(c.t["q"])
        for _ in range(10):
            decode(pa, c, c.t, out, m)
        want.append((out, m))
    torch.cuda.synchronize()
    got = [(torch.empty_like(o), torch.zeros_like(m)) for o, m in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, (o, m) in zip(cases, streams, got):
            decode(pa, c, c.t, o, m, stream=s)
    torch.cuda.synchronize()
    for (o, m), (wo, wm) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(m, wm)


def test_calls_in_a_row_without_synchronisation(pa):
    """Decode, eviction in place and decode again, repeated with lengths that torch operations
    compute on the device between the calls."""
    case = Case(np.random.default_rng(20), [600, 333, 64], 8, 2, 128, 16, "bf16")
    first = {k: v.clone() for k, v in case.t.items()}

    def run(wait):
        t = {k: v.clone() for k, v in first.items()}
        mass = torch.zeros((3, 2, 600), device=dev())
        outs = []
        for keep in (300, 299, 100, 50, 49):
            out = torch.empty_like(t["q"])
            decode(pa, case, t, out, mass, max_context_len=600)
            outs.append(out)
            kp = torch.full((3,), keep, dtype=torch.int32, device=dev())
            kept = torch.empty((3, 2, 300), dtype=torch.int32, device=dev())
            pa.paged_kv_evict(kept, mass, mass, t["kc"], t["vc"], t["bt"], t["bt"], t["lens"], kp, 8,
                              kv_params=t["par"])
            outs.append(kept)
            t["lens"] = torch.minimum(t["lens"], kp)
            if wait:
                torch.cuda.synchronize()
        return outs

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
    assert pa.get_device_error() == 0


# ---------------------------------------------------------------------------- large caches

@pytest.mark.parametrize("int4", [True, False])
def test_offsets_past_32_bits(pa, int4):
    """Rows at the far end of caches of more than 4 GiB (int4) and 8 GiB."""
    d = dev()
    Hk, bs, D, H = 8, 64, 128, 16
    NB = 135000 if int4 else 66000               # 8 * 64 * 64 bytes, or 64 * 8 * 256, a block
    rng = np.random.default_rng(30)
    if int4:
        kc = torch.empty((NB, Hk, bs, D // 2), dtype=torch.uint8, device=d)
        par = torch.empty((NB, Hk, bs, 4), dtype=torch.float16, device=d)
    else:
        kc = torch.empty((NB, bs, Hk, D), dtype=torch.bfloat16, device=d)
        par = None
    vc = torch.empty_like(kc)
    assert kc.numel() * kc.element_size() > 1 << 32
    n, keep = 150, 70
    bt = torch.tensor([[NB - 1, 3, NB - 7]], dtype=torch.int32, device=d)
    obt = torch.tensor([[NB - 2, NB - 3]], dtype=torch.int32, device=d)
    slots = torch.tensor([int(bt[0, t // bs]) * bs + t % bs for t in range(n)], dtype=torch.int32, device=d)
    x_k, x_v = rows(rng, (n, Hk, D), "k"), rows(rng, (n, Hk, D))
    k, v = (torch.from_numpy(x).to(d).bfloat16() for x in (x_k, x_v))
    lens = torch.tensor([n], dtype=torch.int32, device=d)
    q = torch.from_numpy(rng.standard_normal((1, H, D)).astype(np.float32)).to(d).bfloat16()
    out = torch.empty_like(q)
    mass = torch.zeros((1, Hk, n), device=d)
    if int4:
        pa.paged_kv_write_int4(k, v, slots, kc, vc, par)
        pa.paged_attention_decode_int4(out, q, kc, vc, par, bt, lens, D ** -0.5, mass=mass)
        hk, hv = (cc.values(*cc.cache_rows(cc.stored(x, "bf16").astype(np.float32))) for x in (x_k, x_v))
    else:
        pa.paged_kv_write(k, v, slots, kc, vc)
        pa.paged_attention_decode_scored(out, q, mass, kc, vc, bt, lens, D ** -0.5)
        hk, hv = cc.stored(x_k, "bf16"), cc.stored(x_v, "bf16")
    ref, w, _, wv = cc.attention(q[0].double().cpu().numpy(), hk, hv, D ** -0.5)
    # bf16 output and weights: half a step of each, and the sums
    assert (np.abs(out[0].double().cpu().numpy() - ref) <= np.abs(ref) * 2.0 ** -8 + 4 * 2.0 ** -8 * wv).all()
    m = mass[0].cpu().numpy()
    assert np.abs(m - cc.group_mass(w, Hk)).max() <= 1e-3
    kept = torch.empty((1, Hk, keep), dtype=torch.int32, device=d)
    mo = torch.empty((1, Hk, keep), device=d)
    pa.paged_kv_evict(kept, mass, mo, kc, vc, bt, obt, lens, torch.tensor([keep], dtype=torch.int32, device=d), 5,
                      kv_params=par)
    oslots = torch.tensor([int(obt[0, t // bs]) * bs + t % bs for t in range(keep)], dtype=torch.int32, device=d)
    ko = torch.empty((keep, Hk, D), dtype=torch.float32 if int4 else torch.bfloat16, device=d)
    vo = torch.empty_like(ko)
    if int4:
        pa.paged_kv_read_int4(ko, vo, oslots, kc, vc, par)
    else:
        ko, vo = kc.view(-1, Hk, D)[oslots.long()], vc.view(-1, Hk, D)[oslots.long()]
    for h in range(Hk):
        at = cc.evict(m[h], n, keep, 5)
        assert np.array_equal(kept[0, h].cpu().numpy(), at)
        assert np.array_equal(ko[:, h].float().cpu().numpy(), hk[at, h].astype(np.float32))
        assert np.array_equal(vo[:, h].float().cpu().numpy(), hv[at, h].astype(np.float32))
    assert pa.get_device_error() == 0


# ---------------------------------------------------------------------------- the allocator

def test_forked_sequences_evicted_into_new_ones(pa):
    """Forks share their blocks, so each is evicted into blocks of a sequence of its own; the shared
    blocks keep what the sibling reads, and the allocator has them back once both have moved."""
    d = dev()
    Hk, H, bs, D, keep = 2, 8, 16, 128, 20
    rng = np.random.default_rng(40)
    al = pa.BlockAllocator(64, bs)
    al.add_seq(0)
    slots, _ = al.append(0, 100)
    kc = torch.zeros((64, Hk, bs, D // 2), dtype=torch.uint8, device=d)
    vc, par = torch.zeros_like(kc), torch.full((64, Hk, bs, 4), float("nan"), dtype=torch.float16, device=d)
    x_k, x_v = rows(rng, (100, Hk, D), "k"), rows(rng, (100, Hk, D))

    def write(s, a, b):
        pa.paged_kv_write_int4(torch.from_numpy(a).to(d), torch.from_numpy(b).to(d), torch.from_numpy(s).to(d), kc, vc,
                               par)

    write(slots, x_k, x_v)
    held = {0: [cc.values(*cc.cache_rows(x)) for x in (x_k, x_v)]}
    al.fork(0, 1)
    held[1] = [a.copy() for a in held[0]]
    for s in (0, 1):                             # each fork goes on by itself
        a, b = rows(rng, (3, Hk, D), "k"), rows(rng, (3, Hk, D))
        slots, pairs = al.append(s, 3)
        if len(pairs):
            pa.copy_blocks(kc, vc, torch.from_numpy(pairs).to(d), kv_params=par)
        write(slots, a, b)
        held[s] = [np.concatenate((x, cc.values(*cc.cache_rows(y)))) for x, y in zip(held[s], (a, b))]
    q = rng.standard_normal((2, H, D)).astype(np.float32) * np.float32(2.0)
    qd = torch.from_numpy(q).to(d).half()

    def attend(ids, mass):
        bt, lens = al.export(ids, 8)
        out = torch.empty_like(qd)
        pa.paged_attention_decode_int4(out, qd, kc, vc, par, torch.from_numpy(bt).to(d), torch.from_numpy(lens).to(d),
                                       D ** -0.5, mass=mass)
        for i, s in enumerate(ids):
            for h in range(Hk):
                ref, _, _, wv = cc.attention(cc.stored(q[i, 4 * h:4 * h + 4], "f16"), held[s][0][:, h:h + 1],
                                             held[s][1][:, h:h + 1], D ** -0.5)
                # f16 output and weights (2^-11 each of what is summed, at most |value| + 2 |zero|), scores in f32
                assert (np.abs(out[i, 4 * h:4 * h + 4].double().cpu().numpy() - ref) <= 4e-3).all()
        return bt, lens

    mass = torch.zeros((2, Hk, 128), device=d)
    bt, lens = attend([0, 1], mass)
    m = mass.cpu().numpy()
    for s in (2, 3):
        al.add_seq(s)
        al.append(s, keep)
    obt, _ = al.export([2, 3], 8)
    kept = torch.empty((2, Hk, keep), dtype=torch.int32, device=d)
    mo = torch.zeros((2, Hk, 128), device=d)
    pa.paged_kv_evict(kept, mass, mo, kc, vc, torch.from_numpy(bt).to(d), torch.from_numpy(obt).to(d),
                      torch.from_numpy(lens).to(d), torch.full((2,), keep, dtype=torch.int32, device=d), 4,
                      kv_params=par)
    for i, s in enumerate((0, 1)):
        held[s + 2] = [np.stack([x[cc.evict(m[i, h], int(lens[i]), keep, 4), h] for h in range(Hk)], 1)
                       for x in held[s]]
    attend([0, 1], torch.zeros_like(mass))       # the forks still read what they did
    attend([2, 3], mo)
    used = al.stats().num_used
    al.free_seq(0)
    al.free_seq(1)
    assert al.stats().num_used == 2 * -(-keep // bs) < used
    attend([2, 3], mo)
    assert pa.get_device_error() == 0
