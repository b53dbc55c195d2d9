"""A serving step's calls in the ways that a program may make them besides: prompts captured in a graph (the layout's
two launches), from two threads at once, rows without kv heads, single rows of any stride."""
import threading

import numpy as np
import pytest
import torch

import step_cases as sc
from gpu_cases import dev, pa_mod
from test_gpu_fp8_block import RUNS
from test_gpu_rotary import assert_close
from test_gpu_step_run import Loop, plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


@pytest.mark.parametrize("bound", [0, RUNS])
def test_prompts_captured_in_a_graph(pa, bound):
    """Release, append of many tokens, rotation, scatter, decode and read-back in one graph, lengths and height in
    place, replayed over several steps; equal to the same steps run eagerly."""
    def make():
        loop = Loop(pa, 90, 7, 400, T=1500, width=60, bound=bound)
        loop.rows = [torch.zeros((1500, loop.Hk, loop.D), dtype=loop.qkv.dtype, device=dev()) for _ in range(2)]
        return loop

    def step(loop):
        loop.step()
        pa.paged_kv_read_fp8_block(*loop.rows, loop.slots, loop.kc, loop.vc, loop.sc)

    captured, eager = make(), make()
    for loop in (captured, eager):
        loop.feed(np.zeros(7), np.zeros(7))
        step(loop)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(captured)
    rng, held = np.random.default_rng(91), np.zeros(7, int)
    for i in range(6):
        done = (held > 500) | (rng.random(7) < 0.2)
        held[done] = 0
        new = rng.integers(0, 210, 7)
        held += new
        captured.feed(new, done)
        eager.feed(new, done)
        g.replay()
        step(eager)
        for a, b in ((captured.out, eager.out), (captured.kc, eager.kc), (captured.vc, eager.vc), (captured.table, eager.table),
                     (captured.lens, eager.lens), (captured.slots, eager.slots), (captured.pos, eager.pos),
                     (captured.free, eager.free), (captured.num_free, eager.num_free), (captured.qkv, eager.qkv),
                     *zip(captured.rows, eager.rows)):
            assert torch.equal(a, b), i
        assert captured.lens.tolist() == held.tolist()
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("plain", [False, True])
def test_two_threads_at_once(pa, monkeypatch, plain):
    """Two loops, each from a thread and on a stream of its own; equal to the loops run one after the other."""
    if plain:
        monkeypatch.setattr(pa, "_binding", None)

    def run(loop, steps, outs, stream, errors):
        try:
            with torch.cuda.stream(stream):
                for new, done in steps:
                    loop.feed(new, done)
                    loop.step()
                    outs.append(loop.out.clone())
            stream.synchronize()
        except Exception as e:
            errors.append(e)

    def make():
        loops = [Loop(pa, 95 + i, 6, 60, bound=b) for i, b in enumerate((0, RUNS))]
        return [(l, list(plan(np.random.default_rng(97 + i), l, 12)), [], torch.cuda.Stream(), []) for i, l in enumerate(loops)]

    alone, both = make(), make()
    torch.cuda.synchronize()
    for work in alone:
        run(*work)
    threads = [threading.Thread(target=run, args=work) for work in both]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert not a[4] and not b[4]
        assert all(torch.equal(x, y) for x, y in zip(a[2], b[2])) and len(a[2]) == len(b[2]) == 12
        for n in ("kc", "vc", "table", "lens", "free", "num_free", "qkv"):
            assert torch.equal(getattr(a[0], n), getattr(b[0], n)), n
    pa.get_device_error()


@pytest.mark.parametrize("plain", [False, True])
def test_rows_of_no_kv_heads_and_single_rows(pa, monkeypatch, plain):
    """Keys of no heads; one token as a slice whose stride means nothing; the same row for every token."""
    if plain:
        monkeypatch.setattr(pa, "_binding", None)
    rng = np.random.default_rng(99)
    x = rng.standard_normal((5, 4, 64)).astype(np.float32)
    xt, f = torch.from_numpy(x).to(dev()), pa.rotary_frequencies(64)
    pos = np.array([3, 99, 5000, 0, 7], np.int32)
    pt, ft = torch.from_numpy(pos).to(dev()), torch.from_numpy(f).to(dev())
    out = torch.zeros_like(xt)
    none = torch.zeros((5, 0, 64), device=dev())
    pa.rotary_embedding(out, none, xt, none.clone(), pt, ft)
    assert_close(out, x.astype(np.float64), pos, f, 1.0, False, "f32")
    one = torch.zeros((1, 4, 64), device=dev())
    pa.rotary_embedding(one, None, xt[1:2].as_strided((1, 4, 64), (12345, 64, 1)), None, pt[1:2], ft)
    assert torch.equal(one[0], out[1])
    same = xt[2:3].expand(5, 4, 64)
    pa.rotary_embedding(out, None, same, None, pt, ft)
    assert_close(out, np.broadcast_to(x[2], (5, 4, 64)).astype(np.float64), pos, f, 1.0, False, "f32")
    # one token into a block-scaled cache, its row's stride a number that means nothing
    kc, s = torch.zeros((2, 4, 8, 64), dtype=torch.uint8, device=dev()), torch.zeros((2, 4, 2), device=dev())
    vc, hk, hs = kc.clone(), kc.cpu().numpy(), s.cpu().numpy()
    hv = hk.copy()
    row = xt[1:2].as_strided((1, 4, 64), (7, 64, 1))
    want = x[0:1] if xt[1:2].storage_offset() == 0 else x[1:2]
    pa.paged_kv_write_fp8_block(row, row, torch.tensor([8], dtype=torch.int32, device=dev()), kc, vc, s)
    sc.write_blocks(hk, hv, hs, x[1:2].astype(np.float64), x[1:2].astype(np.float64), [8])
    assert sc.same_codes(kc.cpu().numpy(), hk) and sc.same_codes(vc.cpu().numpy(), hv) and np.array_equal(s.cpu().numpy(), hs)
    assert pa.get_device_error() == 0
