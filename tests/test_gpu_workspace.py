"""The binding's own workspaces when a call launches on another stream than the current one,
eagerly and inside a captured graph: every decode call against the same call alone, bit for bit."""
import numpy as np
import pytest
import torch

from gpu_cases import dev, pa_mod

pytestmark = pytest.mark.gpu

H, HK, D, BS = 16, 4, 128, 16


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


class Batch:
    """A cache of random tokens and one decode call over it; several partitions a row."""

    def __init__(self, pa, kind, seed, lens):
        d = dev()
        g = torch.Generator(device=d)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=d)
        self.pa, self.kind, B, width = pa, kind, len(lens), -(-max(lens) // BS)
        NB = B * width
        self.lens = torch.tensor(lens, dtype=torch.int32, device=d)
        self.bt = torch.randperm(NB, generator=g, device=d).to(torch.int32).view(B, width)
        if kind == "shared":                     # the first 512 tokens are the same blocks for every sequence
            self.bt[:, :512 // BS] = self.bt[0, :512 // BS]
            self.prefix = torch.full((B,), 512, dtype=torch.int32, device=d)
            self.groups = torch.arange(B, dtype=torch.int32, device=d).view(1, B)
        self.dtype = torch.float32 if kind == "simt" else torch.bfloat16
        self.q = rand(B, H, D).to(self.dtype)
        self.new = [rand(B, HK, D).to(self.dtype) for _ in range(2)]
        at = self.lens.long() - 1
        self.slots = (self.bt.gather(1, (at // BS)[:, None])[:, 0].long() * BS + at % BS).to(torch.int32)
        x = [rand(NB * BS, HK, D) for _ in range(2)]
        every = torch.arange(NB * BS, dtype=torch.int32, device=d)
        if kind.startswith("int4"):
            self.cache = [torch.zeros((NB, HK, BS, D // 2), dtype=torch.uint8, device=d) for _ in range(2)]
            self.cache.append(torch.zeros((NB, HK, BS, 4), dtype=torch.float16, device=d))
            pa.paged_kv_write_int4(*x, every, *self.cache)
        elif kind.startswith("fp8"):
            self.cache = [torch.zeros((NB, BS, HK, D), dtype=torch.uint8, device=d) for _ in range(2)]
            pa.paged_kv_write_fp8(*x, every, *self.cache, 0.02, 0.02)
        else:
            self.cache = [a.to(self.dtype).view(NB, BS, HK, D) for a in x]
        self.out, self.mass = torch.empty_like(self.q), torch.zeros((B, HK, width * BS), device=d)

    def call(self, **kw):
        pa, c, scale = self.pa, self.cache, D ** -0.5
        head, tail = (self.out, self.q), (self.bt, self.lens)
        if self.kind in ("plain", "simt"):
            pa.paged_attention_decode(*head, *c, *tail, scale, **kw)
        elif self.kind == "append":
            pa.paged_attention_decode_append(*head, *self.new, self.slots, *c, *tail, scale, **kw)
        elif self.kind == "shared":
            pa.paged_attention_decode_shared(*head, *c, *tail, self.prefix, self.groups, scale, **kw)
        elif self.kind == "fp8":
            pa.paged_attention_decode_fp8(*head, *c, *tail, scale, 0.02, 0.02, **kw)
        elif self.kind == "fp8_append":
            pa.paged_attention_decode_fp8_append(*head, *self.new, self.slots, *c, *tail, scale, 0.02, 0.02, **kw)
        elif self.kind == "scored":
            pa.paged_attention_decode_scored(*head, self.mass, *c, *tail, scale, **kw)
        else:
            pa.paged_attention_decode_int4(*head, *c, *tail, scale, mass=self.mass if self.kind == "int4_mass" else None,
                                           **kw)

    def clear(self):
        self.out.fill_(float("nan"))
        self.mass.zero_()

    def alone(self, calls):
        """What `calls` calls in a row give through a workspace of their own."""
        self.clear()
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=dev())
        for _ in range(calls):
            self.call(workspace=ws)
        torch.cuda.synchronize()
        return self.out.clone(), self.mass.clone()


KINDS = ["plain", "simt", "append", "shared", "fp8", "fp8_append", "int4", "int4_mass", "scored"]


@pytest.fixture
def handed(pa, monkeypatch):
    """Every workspace handed out: (stream, first byte, byte past the last)."""
    seen, inner = [], pa._workspace

    def spy(device, stream_ptr, nbytes):
        buf = inner(device, stream_ptr, nbytes)
        seen.append((stream_ptr, buf.data_ptr(), buf.data_ptr() + buf.numel()))
        return buf

    monkeypatch.setattr(pa, "_workspace", spy)
    return seen


def assert_apart(handed, streams):
    assert {s for s, _, _ in handed} == {s.cuda_stream for s in streams}
    for s, a, b in handed:
        for t, c, d in handed:
            assert s == t or b <= c or d <= a


@pytest.mark.parametrize("kind", KINDS)
def test_two_branches_of_one_graph(pa, handed, kind):
    """One capture forks: calls go to a side stream through stream=, others and torch operations that
    allocate run beside them on the capture's own stream. Replays equal the calls run alone."""
    a, b = Batch(pa, kind, 1, [2500, 900, 1300, 1700]), Batch(pa, kind, 2, [1100, 3000, 2049])
    want = [x.alone(4) for x in (a, b)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        for _ in range(4):
            a.call(stream=side)
            junk = torch.full((8 << 20,), 255, dtype=torch.uint8, device=dev())
            b.call()
            junk = junk + 1
        cur.wait_stream(side)
    assert_apart(handed, (cur, side))
    for _ in range(5):
        a.clear()
        b.clear()
        g.replay()
        torch.cuda.synchronize()
        for x, (out, mass) in zip((a, b), want):
            assert torch.equal(x.out, out) and torch.equal(x.mass, mass)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("default", [False, True], ids=["side", "default"])
@pytest.mark.parametrize("kind", ["plain", "int4_mass", "scored"])
def test_eager_calls_on_another_stream(pa, handed, kind, default):
    """stream= names a side stream, or the default one while a side stream is current; torch operations on
    the current stream allocate and write beside the calls."""
    a = Batch(pa, kind, 3, [2500, 900, 1300, 1700])
    out, mass = a.alone(4)
    side = torch.cuda.Stream()
    other, cur = (torch.cuda.default_stream(), side) if default else (side, torch.cuda.current_stream())
    a.clear()
    torch.cuda.synchronize()
    pa._ws_cache.clear()
    with torch.cuda.stream(cur):
        for _ in range(4):
            junk = torch.full((8 << 20,), 255, dtype=torch.uint8, device=dev())
            del junk
            a.call(stream=other)
            junk = torch.full((8 << 20,), 255, dtype=torch.uint8, device=dev())
        assert torch.cuda.current_stream() == cur
    torch.cuda.synchronize()
    assert {s for s, _, _ in handed} == {other.cuda_stream}
    assert torch.equal(a.out, out) and torch.equal(a.mass, mass)
    assert pa.get_device_error() == 0


def test_a_captured_stream_that_is_not_current(pa):
    """A call captured through stream= while the current stream is not has memory of the graph's: an eager
    call that grows that stream's cached buffer must not take it from under the graph."""
    a, b = Batch(pa, "scored", 4, [2500, 900]), Batch(pa, "scored", 5, [3000] * 24)
    (out, mass), (out_b, mass_b) = a.alone(1), b.alone(1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a.call()                                 # the stream's cached buffer, of a's size
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    main = torch.cuda.current_stream()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(main):
            a.call(stream=s)
    with torch.cuda.stream(s):
        b.clear()
        b.call()                                 # a larger one
        junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=dev()) for _ in range(64)]
    a.clear()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, out) and torch.equal(a.mass, mass) and len(junk) == 64
    assert torch.equal(b.out, out_b) and torch.equal(b.mass, mass_b)
    assert pa.get_device_error() == 0
