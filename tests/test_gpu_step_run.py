"""A serving loop's steps over a block-scaled 8-bit cache, as they would be used together: blocks given back
and taken on the GPU, queries and keys rotated, keys and values stored, the cache attended and read back;
eagerly, captured in graphs, on two streams, and beside the host allocator's forks."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import compress_cases as cc
import step_cases as sc
from gpu_cases import dev, pa_mod
from test_gpu_fp8_block import RUNS, expected

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


class Loop:
    """Requests in B rows of one table over a pool of NB blocks; every tensor of a step lives here."""

    def __init__(self, pa, seed, B, NB, H=8, Hk=2, D=128, bs=16, T=96, width=20, dtype="bf16", inter=False,
                 bound=0):
        self.bound = bound                           # on the contexts: 0 the table's width, or RUNS
        self.pa, self.B, self.NB, self.H, self.Hk, self.D, self.bs, self.T = pa, B, NB, H, Hk, D, bs, T
        self.dtype, self.inter, self.rng, self.scale = dtype, inter, np.random.default_rng(seed), D ** -0.5
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev())
        self.table, self.lens, self.new = i32(B, width) - 1, i32(B), i32(B)
        self.free = torch.from_numpy(self.rng.permutation(NB).astype(np.int32)).to(dev())
        self.num_free = i32(1) + NB
        self.done = torch.zeros(B, dtype=torch.bool, device=dev())
        self.start, self.slots, self.pos = i32(B + 1), i32(T), i32(T)
        self.kc = torch.from_numpy(self.rng.integers(0, 256, (NB, Hk, bs, D), dtype=np.uint8)).to(dev())
        self.vc, self.sc = self.kc.clone(), torch.full((NB, Hk, 2), float("nan"), device=dev())
        self.qkv = torch.zeros((T, H + 2 * Hk, D), dtype=cc.TORCH[dtype], device=dev())
        self.f = pa.rotary_frequencies(D // 2, scaling="by_turns", scale=4.0)
        self.freq = torch.from_numpy(self.f).to(dev())
        self.q = torch.zeros((B, H, D), dtype=cc.TORCH[dtype], device=dev())
        self.out = torch.zeros_like(self.q)
        self.last = torch.zeros(B, dtype=torch.long, device=dev())

    def step(self, stream=None):
        """One step: what a captured graph holds."""
        pa = self.pa
        q, k, v = self.qkv[:, :self.H], self.qkv[:, self.H:self.H + self.Hk], self.qkv[:, self.H + self.Hk:]
        kw = dict(stream=stream)
        pa.paged_blocks_release(self.table, self.lens, self.done, self.free, self.num_free, self.bs, **kw)
        pa.paged_blocks_append(self.table, self.lens, self.new, self.free, self.num_free, self.start, self.slots, self.pos,
                               self.bs, self.NB, **kw)
        pa.rotary_embedding(q, k, q, k, self.pos, self.freq, interleaved=self.inter, **kw)
        pa.paged_kv_write_fp8_block(k, v, self.slots, self.kc, self.vc, self.sc, **kw)
        # the queries of every request's last token
        if stream is None:
            torch.index_select(q, 0, (self.start[1:].long() - 1).clamp(min=0), out=self.q)
        pa.paged_attention_decode_fp8_block(self.out, self.q, self.kc, self.vc, self.sc, self.table, self.lens,
                                            self.scale, max_context_len=self.bound, **kw)

    def feed(self, new, done):
        """The next step's inputs, written in place; their host copies."""
        x = self.rng.standard_normal(tuple(self.qkv.shape)).astype(np.float32)
        x[::5] *= 4
        self.qkv.copy_(torch.from_numpy(x).to(dev()))
        self.new.copy_(torch.from_numpy(np.asarray(new, np.int32)))
        self.done.copy_(torch.from_numpy(np.asarray(done, bool)))
        return cc.stored(x, self.dtype)


class Model:
    """The loop's plain double: a list of every request's rotated keys and values, as the cache would hold them."""

    def __init__(self, loop):
        self.l = loop
        self.table, self.lens = loop.table.cpu().numpy(), loop.lens.cpu().numpy()
        self.free, self.nf = loop.free.cpu().numpy(), int(loop.num_free)
        self.kc, self.vc, self.sc = (t.cpu().numpy() for t in (loop.kc, loop.vc, loop.sc))
        self.err = set()

    def layout(self, new, done):
        """The step's tables and maps, checked whole numbers for whole numbers."""
        l = self.l
        self.lens, self.free, self.nf, e1 = sc.release(self.table, self.lens, done, self.free, self.nf, l.bs, l.NB)
        self.table, self.lens, self.nf, start, slots, pos, e2 = sc.append(
            self.table, self.lens, np.asarray(new, np.int32), self.free, self.nf, l.T, l.bs, l.NB)
        self.err |= e1 | e2
        for t, w in ((l.table, self.table), (l.lens, self.lens), (l.start, start), (l.slots, slots), (l.pos, pos)):
            assert np.array_equal(t.cpu().numpy(), w)
        assert int(l.num_free) == self.nf and np.array_equal(l.free.cpu().numpy()[:self.nf], self.free[:self.nf])
        return start, slots, pos

    def check(self, x, new, done):
        """After a step whose projection was x: rotation, cache and attention."""
        l = self.l
        start, slots, pos = self.layout(new, done)
        n = int(start[-1])
        # the rotated projection, as stored; the library's own rounding from here on
        got = l.qkv.double().cpu().numpy()
        for a, b in ((0, l.H), (l.H, l.H + l.Hk)):
            ref = sc.rotate(x[:, a:b], pos, l.f, 1.0, l.inter)
            tol = sc.rotate_bound(x[:, a:b], ref, pos, l.f, 1.0, l.inter, cc.EPS[l.dtype])
            assert (np.abs(got[:, a:b] - ref) <= tol)[:n].all()
        k, v = got[:, l.H:l.H + l.Hk], got[:, l.H + l.Hk:]
        assert np.array_equal(v, x[:, l.H + l.Hk:])
        sc.write_blocks(self.kc, self.vc, self.sc, k, v, slots)
        assert sc.same_codes(l.kc.cpu().numpy(), self.kc) and sc.same_codes(l.vc.cpu().numpy(), self.vc)
        assert np.array_equal(l.sc.cpu().numpy(), self.sc, equal_nan=True)
        q, out = l.q.double().cpu().numpy(), l.out.double().cpu().numpy()
        for b, c in enumerate(self.lens):
            t = np.arange(c)
            blk, off = self.table[b, t // l.bs], t % l.bs
            kb, vb = (sc.E4M3[cache[blk, :, off]] * self.sc[blk, :, i].astype(np.float64)[..., None]
                      for i, cache in enumerate((self.kc, self.vc)))
            ref, tol = expected(q[b], kb, vb, l.scale, l.dtype)
            assert (np.abs(out[b] - ref) <= tol).all(), b


def plan(rng, loop, steps, room=96):
    """New tokens and finished requests of some steps: prompts, single tokens, idle rows."""
    held = np.zeros(loop.B, int)
    for _ in range(steps):
        done = (held > 0) & (rng.random(loop.B) < 0.15)
        held[done] = 0
        new = np.where(held == 0, rng.integers(0, 60, loop.B), rng.integers(0, 2, loop.B))
        new = np.where(np.cumsum(new) <= room, new, 0)
        held += new
        yield new.astype(np.int32), done


@pytest.mark.parametrize("dtype,D,bs,inter", [("bf16", 128, 16, False), ("f16", 64, 8, True), ("bf16", 128, 64, True)])
def test_steps_against_plain_forms(pa, dtype, D, bs, inter):
    loop = Loop(pa, 1, 6, 300 // bs + 6, D=D, bs=bs, width=400 // bs, dtype=dtype, inter=inter)
    model = Model(loop)
    for new, done in plan(np.random.default_rng(2), loop, 14):
        x = loop.feed(new, done)
        loop.step()
        model.check(x, new, done)
    code = {"free": pa.PA_DEVERR_FREE_BLOCKS, "context": pa.PA_DEVERR_CONTEXT}
    assert pa.get_device_error() == sum(code[e] for e in model.err)


@pytest.mark.parametrize("bound", [0, RUNS])
def test_steps_without_synchronisation(pa, bound):
    """The same steps enqueued in one go, and with a wait after every call, leave the same caches."""
    def run(wait):
        loop = Loop(pa, 3, 6, 40, bound=bound)
        outs = []
        for new, done in plan(np.random.default_rng(4), loop, 10):
            loop.feed(new, done)
            loop.step()
            outs.append(loop.out.clone())
            if wait:
                torch.cuda.synchronize()
        return outs + [loop.kc, loop.vc, torch.nan_to_num(loop.sc), loop.table, loop.lens, loop.free, loop.num_free]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
    pa.get_device_error()


@pytest.mark.parametrize("bound", [0, RUNS])
def test_two_graphs_replayed_in_turn(pa, bound):
    """Two loops' steps captured, replayed in turn with new inputs written in place, beside the same steps run
    eagerly; the first graph is destroyed before the second runs on."""
    loops, twins = ([Loop(pa, 10 + i, B, NB, H=H, Hk=2, bound=bound) for i, (B, NB, H) in enumerate(((5, 40, 8), (9, 60, 24)))]
                    for _ in range(2))
    plans = [list(plan(np.random.default_rng(20 + i), l, 8)) for i, l in enumerate(loops)]
    for l, t in zip(loops, twins):               # warm up without new tokens
        for x in (l, t):
            x.feed(np.zeros(x.B), np.zeros(x.B))
            x.step()
    torch.cuda.synchronize()
    graphs = []
    for l in loops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l.step()
        graphs.append(g)
    for i in range(8):
        for j, (l, t) in enumerate(zip(loops, twins)):
            if graphs[j] is None:
                continue
            l.feed(*plans[j][i])
            t.feed(*plans[j][i])
            graphs[j].replay()
            t.step()
            for a, b in ((l.out, t.out), (l.kc, t.kc), (l.vc, t.vc), (l.table, t.table), (l.lens, t.lens),
                         (l.slots, t.slots), (l.free, t.free), (l.num_free, t.num_free), (l.qkv, t.qkv)):
                assert torch.equal(a, b), (i, j)
        if i == 3:
            graphs[0].reset()
            graphs[0] = None
            torch.cuda.empty_cache()
    pa.get_device_error()


@pytest.mark.parametrize("bound", [0, RUNS])
def test_two_streams_at_once(pa, bound):
    """Steps of two loops on two streams through stream=, their queries given; equal to the steps run alone."""
    def make():
        loops = [Loop(pa, 30 + i, B, NB, bound=bound) for i, (B, NB) in enumerate(((4, 40), (7, 60)))]
        for l in loops:
            l.q.copy_(torch.from_numpy(np.random.default_rng(5).standard_normal(tuple(l.q.shape)).astype(np.float32)))
            l.feed(np.minimum(np.arange(l.B) * 7 + 1, 96 // l.B), np.zeros(l.B))
        return loops

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone, both = make(), make()
    torch.cuda.synchronize()
    for l, s in zip(alone, streams):
        for _ in range(6):
            l.step(stream=s)
        torch.cuda.synchronize()
    for _ in range(6):
        for l, s in zip(both, streams):
            l.step(stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for x, y in ((a.out, b.out), (a.kc, b.kc), (a.lens, b.lens), (a.slots, b.slots), (a.qkv, b.qkv)):
            assert torch.equal(x, y)
    pa.get_device_error()


def test_lengths_and_decode_next_to_each_other(pa):
    """A decode right after the lengths were made, over and over: it sees the new ones (many tokens, whose lengths
    a second launch writes, and few)."""
    for T, n in ((96, 1), (20000, 900)):
        B, bs, Hk, D = 8, 16, 2, 128
        NB, width = 4000, 600
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev())
        table, lens, free = i32(B, width), i32(B), torch.arange(NB, dtype=torch.int32, device=dev())
        nf, new = i32(1) + NB, i32(B) + n
        kc = torch.full((NB, Hk, bs, D), 0x38, dtype=torch.uint8, device=dev())      # ones
        vs = torch.zeros((NB, Hk, 2), device=dev())
        vs[..., 0] = 1e-3
        q = torch.zeros((B, 4, D), dtype=torch.bfloat16, device=dev())
        outs, start, slots, pos = [], i32(B + 1), i32(T), i32(T)
        # a V block stands for its number's square root; with flat weights the output is the context's mean
        vs[..., 1] = torch.arange(NB, device=dev()).float().sqrt()[:, None]
        for i in range(8):
            pa.paged_blocks_append(table, lens, new, free, nf, start, slots, pos, bs, NB)
            out = torch.empty_like(q)
            pa.paged_attention_decode_fp8_block(out, q, kc, kc, vs, table, lens, 1.0, max_context_len=i % 2 * RUNS)
            outs.append(out)
        torch.cuda.synchronize()
        tab = table.cpu().numpy()
        for i, out in enumerate(outs):
            c = n * (i + 1)
            for b in range(B):
                want = np.sqrt(tab[b, np.arange(c) // bs].astype(np.float64)).mean()
                # bf16 output, weights of 11 bits, float32 sums
                assert abs(float(out[b, 0, 0]) - want) <= want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16)
        assert pa.get_device_error() == 0


def test_forks_of_the_host_allocator(pa):
    """Forked sequences append to a shared, partly filled block: copy-on-write takes codes and scales along, and each
    goes on by itself."""
    Hk, H, bs, D, NB = 2, 8, 16, 128, 16
    rng = np.random.default_rng(40)
    al = pa.BlockAllocator(NB, bs)
    kc = torch.zeros((NB, Hk, bs, D), dtype=torch.uint8, device=dev())
    vc, s = torch.zeros_like(kc), torch.full((NB, Hk, 2), float("nan"), device=dev())
    hk, hv, hs = kc.cpu().numpy(), vc.cpu().numpy(), s.cpu().numpy()

    def write(slots, size):
        x = [rng.standard_normal((len(slots), Hk, D)).astype(np.float32) * np.float32(size) for _ in range(2)]
        pa.paged_kv_write_fp8_block(*(torch.from_numpy(a).to(dev()) for a in x), torch.from_numpy(slots).to(dev()), kc, vc, s)
        sc.write_blocks(hk, hv, hs, x[0].astype(np.float64), x[1].astype(np.float64), slots)

    al.add_seq(0)
    slots, _ = al.append(0, 25)
    write(slots, 1.0)
    al.fork(0, 1)
    for seq, size in ((0, 50.0), (1, 0.01)):     # one outgrows the shared block's scale, the other does not
        slots, pairs = al.append(seq, 3)
        if len(pairs):
            pa.copy_blocks(kc, vc, torch.from_numpy(pairs).to(dev()), kv_scales=s)
            for a, b in pairs:
                hk[b], hv[b], hs[b] = hk[a], hv[a], hs[a]
        write(slots, size)
    assert sc.same_codes(kc.cpu().numpy(), hk) and sc.same_codes(vc.cpu().numpy(), hv)
    assert np.array_equal(s.cpu().numpy(), hs, equal_nan=True)
    bt, lens = al.export([0, 1], 4)
    q = rng.standard_normal((2, H, D)).astype(np.float32)
    qd = torch.from_numpy(q).to(dev()).half()
    out = torch.empty_like(qd)
    pa.paged_attention_decode_fp8_block(out, qd, kc, vc, s, torch.from_numpy(bt).to(dev()), torch.from_numpy(lens).to(dev()),
                                        D ** -0.5)
    for b in range(2):
        t = np.arange(lens[b])
        blk, off = bt[b, t // bs], t % bs
        k, v = (sc.E4M3[c[blk, :, off]] * hs[blk, :, i].astype(np.float64)[..., None] for i, c in enumerate((hk, hv)))
        ref, tol = expected(cc.stored(q[b], "f16"), k, v, D ** -0.5, "f16")
        assert (np.abs(out[b].double().cpu().numpy() - ref) <= tol).all()
    assert pa.get_device_error() == 0


def test_context_read_back_for_prefill(pa):
    """A cached context expanded to 16 bits and attended by the prefill of its next chunk, against the 64-bit form."""
    rng = np.random.default_rng(50)
    Hk, H, bs, D, c, n = 2, 8, 16, 128, 150, 40
    NB = 12
    kc = torch.zeros((NB, Hk, bs, D), dtype=torch.uint8, device=dev())
    vc, s = torch.zeros_like(kc), torch.zeros((NB, Hk, 2), device=dev())
    x = [torch.from_numpy(rng.standard_normal((c, Hk, D)).astype(np.float32)).to(dev()).bfloat16() for _ in range(2)]
    slots = torch.randperm(NB * bs, device=dev())[:0].to(torch.int32)
    table = torch.from_numpy(rng.permutation(NB)[:-(-c // bs)].astype(np.int32)).to(dev())
    t = torch.arange(c, device=dev())
    slots = (table[t // bs] * bs + t % bs).to(torch.int32)
    pa.paged_kv_write_fp8_block(*x, slots, kc, vc, s)
    wide = [torch.zeros((NB, bs, Hk, D), dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    rows = [torch.empty((c, Hk, D), dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    pa.paged_kv_read_fp8_block(*rows, slots, kc, vc, s)
    for w, r in zip(wide, rows):
        w.view(-1, Hk, D)[slots.long()] = r
    q = torch.from_numpy(rng.standard_normal((n, H, D)).astype(np.float32)).to(dev()).bfloat16()
    out = torch.empty_like(q)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    pa.paged_attention_prefill(out, q, *wide, table[None].contiguous(), i32([c]), i32([0, n]), D ** -0.5, n)
    k, v = (r.double().cpu().numpy() for r in rows)
    for i in range(n):
        ref, w, _, wv = cc.attention(q[i].double().cpu().numpy(), k[:c - n + i + 1], v[:c - n + i + 1], D ** -0.5)
        # bf16 output, and weights rounded to bf16 on both sides of the quotient
        assert (np.abs(out[i].double().cpu().numpy() - ref) <= np.abs(ref) * 2.0 ** -8 + 3 * 2.0 ** -8 * wv).all()
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("bound", [0, RUNS])
@pytest.mark.parametrize("plain", [False, True])
def test_two_branches_of_one_graph(pa, monkeypatch, plain, bound):
    """One capture forks: decodes go to a side stream through stream=, others and torch operations that allocate run
    beside them on the capture's own stream; replays equal the calls alone, whichever way the calls go."""
    from test_gpu_fp8_block import Case
    cases = [Case(np.random.default_rng(60 + i), lens, 16, 4, 128, 16, "f16") for i, lens in
             enumerate(([2500, 900, 1300], [1100, 3000, 2049, 5]))]
    want = [c.run(pa, max_context_len=bound) for c in cases]
    seen, inner = [], pa._workspace

    def spy(device, stream_ptr, nbytes):
        buf = inner(device, stream_ptr, nbytes)
        seen.append((stream_ptr, buf.data_ptr(), buf.data_ptr() + buf.numel()))
        return buf

    monkeypatch.setattr(pa, "_workspace", spy)
    if plain:
        monkeypatch.setattr(pa, "_binding", None)
    outs = [torch.empty_like(w) for w in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        for _ in range(4):
            cases[0].run(pa, out=outs[0], stream=side, max_context_len=bound)
            junk = torch.full((8 << 20,), 255, dtype=torch.uint8, device=dev())
            cases[1].run(pa, out=outs[1], max_context_len=bound)
            junk = junk + 1
        cur.wait_stream(side)
    # a stream that is not the current one is the Python code's affair
    assert {s for s, _, _ in seen} == ({cur.cuda_stream, side.cuda_stream} if plain else {side.cuda_stream})
    for s, a, b in seen:
        for t, c, d in seen:
            assert s == t or b <= c or d <= a
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert pa.get_device_error() == 0


def test_python_code_and_compiled_way_agree(pa, monkeypatch):
    """The steps through the compiled module and through the Python code alone leave the same tensors; what the
    module does not take, as a tensor subclass's rows that are not dense, the Python code refuses."""
    def run(plain):
        if plain:
            monkeypatch.setattr(pa, "_binding", None)
        loop = Loop(pa, 70, 6, 40)
        store = Loop(pa, 71, 3, 20)
        cache = [torch.zeros((20, 16, 2, 128), dtype=torch.bfloat16, device=dev()) for _ in range(2)]
        rows = [torch.zeros((96, 2, 128), dtype=torch.bfloat16, device=dev()) for _ in range(2)]
        for new, done in plan(np.random.default_rng(72), loop, 6):
            loop.feed(new, done)
            loop.step()
            store.feed(new[:3], done[:3])
            pa.paged_blocks_append(store.table, store.lens, store.new, store.free, store.num_free, store.start,
                                   store.slots, store.pos, 16, 20)
            q, k, v = store.qkv[:, :8], store.qkv[:, 8:10], store.qkv[:, 10:]
            pa.paged_kv_write_rotary(q, q, k, v, store.pos, store.freq, store.slots, *cache, factor=1.5)
            pa.paged_kv_read_fp8_block(*rows, loop.slots, loop.kc, loop.vc, loop.sc)
        pa.get_device_error()
        return [loop.out, loop.kc, loop.vc, loop.table, loop.lens, loop.free, loop.qkv, store.qkv, *cache, *rows]

    assert pa._binding is not None
    a = run(False)
    for x, y in zip(a, run(True)):
        assert torch.equal(x, y)


def test_refusals_are_the_same_both_ways(pa, monkeypatch):
    """Statuses of the library and the Python code's errors, with and without the compiled module."""
    d = dev()
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device=d)
    c = torch.zeros((4, 2, 16, 128), dtype=torch.uint8, device=d)
    s, i = torch.zeros((4, 2, 2), device=d), torch.zeros(4, dtype=torch.int32, device=d)
    one, t = torch.zeros(1, dtype=torch.int32, device=d), torch.zeros((4, 3), dtype=torch.int32, device=d)
    f = torch.zeros(64, dtype=torch.float64, device=d)
    cases = [
        (ValueError, lambda: pa.paged_kv_write_fp8_block(x[:3], x, i, c, c, s)),
        (TypeError, lambda: pa.paged_kv_write_fp8_block(x.double(), x.double(), i, c, c, s)),
        (TypeError, lambda: pa.paged_kv_write_fp8_block(x, x, i, x.view(1, 4, 2, 128), x.view(1, 4, 2, 128), s)),
        (TypeError, lambda: pa.paged_kv_write_fp8_block(x, x, i.long(), c, c, s)),
        (ValueError, lambda: pa.paged_kv_write_fp8_block(x, x, i, c, c, s[:2])),
        (ValueError, lambda: pa.paged_kv_write_fp8_block(x, x.cpu(), i, c, c, s)),
        (ValueError, lambda: pa.paged_kv_read_fp8_block(x.transpose(0, 1), x, i, c, c, s)),
        (pa.PagedAttnError, lambda: pa.paged_kv_write_fp8_block(x[..., :96].contiguous(), x[..., :96].contiguous(), i,
                                                              c[..., :96].contiguous(), c[..., :96].contiguous(), s)),
        (ValueError, lambda: pa.paged_attention_decode_fp8_block(x, x, c, c, s, t, i[:3], 1.0)),
        (ValueError, lambda: pa.paged_attention_decode_fp8_block(x, x, c, c, s, t, i, 1.0, max_context_len=-1)),
        (pa.PagedAttnError, lambda: pa.paged_attention_decode_fp8_block(x, x, c, c, s, t, i, float("nan"))),
        (pa.PagedAttnError, lambda: pa.paged_attention_decode_fp8_block(x.float(), x.float(), c, c, s, t, i, 1.0)),
        (TypeError, lambda: pa.paged_attention_decode_fp8_block(x, x, c, c, s, t, i, 1.0, workspace=s)),
        (pa.PagedAttnError, lambda: pa.rotary_embedding(x, None, x, None, i, f[:12])),
        (ValueError, lambda: pa.rotary_embedding(x, None, x, x, i, f)),
        (TypeError, lambda: pa.rotary_embedding(x.float(), None, x, None, i, f)),
        (ValueError, lambda: pa.paged_kv_write_rotary(x, x, x, x, i, f, i, x, x)),
        (pa.PagedAttnError, lambda: pa.paged_blocks_append(t, i, i, i, one, torch.zeros(5, dtype=torch.int32, device=d), i,
                                                          i, 12, 4)),
        (ValueError, lambda: pa.paged_blocks_append(t, i, i, i, i, i, i, i, 16, 4)),
        (TypeError, lambda: pa.paged_blocks_release(t, i, i, i, one, 16)),
        (pa.PagedAttnError, lambda: pa.paged_blocks_release(t, i, i.bool(), i, one, 16, num_blocks=0)),
    ]
    for _ in range(2):
        for exc, call in cases:
            with pytest.raises(exc):
                call()
        # what is left open works: empty calls, a given stream, flags as numbers
        pa.paged_kv_write_fp8_block(x[:0], x[:0], i[:0], c, c, s)
        pa.rotary_embedding(x, x, x, x, i, f, 1, 1, stream=torch.cuda.current_stream())
        pa.paged_blocks_release(t, i, i.to(torch.uint8), i, one, 16)
        monkeypatch.setattr(pa, "_binding", None)
    assert pa.get_device_error() == 0


FIRST_CALLS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
from test_gpu_step_run import Loop, Model, plan
import paged_kv_cache_261_gb300 as pa
loop = Loop(pa, 30, 5, 40)
model = Model(loop)
steps = list(plan(np.random.default_rng(31), loop, 3))
x = loop.feed(*steps[0])
torch.index_select(loop.q, 0, loop.last)             # torch's own first calls
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    loop.step()
for i, (new, done) in enumerate(steps):
    if i:
        x = loop.feed(new, done)
    g.replay()
    model.check(x, new, done)
"""


def test_first_calls_of_a_process_are_captured(pa):
    """What the library asks the device once (kernels' shared memory, how many clusters have room) may be asked
    inside a capture."""
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
