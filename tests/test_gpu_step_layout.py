"""Block tables and slot maps from lengths on the GPU against request-by-request plain forms: whole
numbers, all equal."""
import numpy as np
import pytest
import torch

import step_cases as sc
from gpu_cases import dev, pa_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def t32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(dev())


def bits(pa, kinds):
    code = {"free": pa.PA_DEVERR_FREE_BLOCKS, "context": pa.PA_DEVERR_CONTEXT, "block": pa.PA_DEVERR_BLOCK_ID}
    return sum(code[k] for k in kinds)


def run_append(pa, table, lens, new, free, nf, T, bs, NB, in_place=False):
    """The call on fresh tensors checked against the plain form; returns what it leaves."""
    want = sc.append(table, lens, new, free, nf, T, bs, NB)
    bt, cl, fr, n = t32(table), t32(lens), t32(free), t32([nf])
    start, slots, pos = (torch.full((m,), 77, dtype=torch.int32, device=dev()) for m in (len(lens) + 1, T, T))
    ncl, nn = (cl, n) if in_place else (torch.full_like(cl, 77), torch.full_like(n, 77))
    kw = {} if in_place else dict(new_context_lens=ncl, new_num_free=nn)
    pa.paged_blocks_append(bt, cl, t32(new), fr, n, start, slots, pos, bs, NB, **kw)
    got = [x.cpu().numpy() for x in (bt, ncl, nn, start, slots, pos)]
    for g, w in zip(got, want):
        assert np.array_equal(g, np.atleast_1d(w))
    assert pa.get_device_error() == bits(pa, want[6])
    assert np.array_equal(fr.cpu().numpy(), free)
    if not in_place:
        assert np.array_equal(cl.cpu().numpy(), lens) and int(n) == nf
    return want


def pool(rng, lens, MB, bs, spare):
    """Tables of lens, and a stack of `spare` free blocks with junk above it."""
    need = [-(-int(n) // bs) for n in lens]
    NB = sum(need) + spare + 1
    perm = rng.permutation(NB).astype(np.int32)
    table, at = np.full((len(lens), MB), -1, np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    free = np.full(NB, 12345, np.int32)
    free[:spare] = perm[at:at + spare]
    return table, free, NB


CASES = [  # requests, longest context, longest query, block size
    (1, 0, 1, 16), (1, 3, 1, 1), (64, 4096, 1, 16), (7, 100, 40, 8), (33, 50, 600, 256), (1, 0, 9000, 16),
    (300, 700, 90, 32), (1024, 200, 30, 16), (1500, 64, 2, 4), (5000, 20, 3, 2), (16384, 5, 2, 4)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,ctx,q,bs", CASES)
def test_append(pa, B, ctx, q, bs, in_place):
    rng = np.random.default_rng(B + ctx)
    lens = rng.integers(0, ctx + 1, B).astype(np.int32)
    new = rng.integers(0, q + 1, B).astype(np.int32)
    new[0] = max(new[0], 1)
    MB = -(-(ctx + q) // bs)
    table, free, NB = pool(rng, lens, MB, bs, B * (q // bs + 1))
    run_append(pa, table, lens, new, free, B * (q // bs + 1), int(new.sum()) + 5, bs, NB, in_place)


@pytest.mark.parametrize("spare", [0, 1, 17, 60])
def test_append_from_a_short_stack(pa, spare):
    """Requests that need no block are served after the stack ran dry, others no more (60 blocks are enough)."""
    rng = np.random.default_rng(spare)
    B, bs, MB = 90, 8, 12
    lens, new = rng.integers(0, 60, B).astype(np.int32), rng.integers(0, 12, B).astype(np.int32)
    table, free, NB = pool(rng, lens, MB, bs, spare)
    want = run_append(pa, table, lens, new, free, spare, int(new.sum()) + 3, bs, NB)
    served = want[1] != lens
    assert (want[6] == {"free"} and served.any() and (new[~served] > 0).any()) if spare < 60 else not want[6]


def test_append_lengths_out_of_range(pa):
    """Negative lengths, contexts past the table, tokens past the outputs, a stack height out of range, bad ids."""
    rng = np.random.default_rng(9)
    lens = np.array([5, -1, 30, 7, 0, 12, 2 ** 31 - 1, 31, 4], np.int32)
    new = np.array([2, 3, 4, -2, 6, 2 ** 31 - 1, 1, 1, 3], np.int32)
    table, free, NB = pool(rng, [5, 0, 30, 7, 0, 12, 0, 31, 4], 4, 8, 9)
    run_append(pa, table, lens, new, free, 9, 40, 8, NB)            # the sixth takes all rows that are left
    new[5] = 4
    for T in (0, 1, 5, 14, 15, 16, 17, 18, 40):
        run_append(pa, table, lens, new, free, 9, T, 8, NB)
    for nf in (-1, len(free) + 1, 2 ** 31 - 1):
        run_append(pa, table, lens, new, free, nf, 40, 8, NB)
    free[7], free[8] = -3, NB
    table[0, 0] = NB + 5
    run_append(pa, table, lens, new, free, 9, 40, 8, NB)
    run_append(pa, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32), free, 9, 3, 8, NB)
    run_append(pa, table[:2], np.array([0, 0], np.int32), np.array([0, 0], np.int32), np.zeros(0, np.int32), 0, 2, 8, NB)


def run_release(pa, table, lens, fin, free, nf, bs, NB, in_place=False):
    want = sc.release(table, lens, fin, free, nf, bs, NB)
    bt, cl, fr, n = t32(table), t32(lens), t32(free), t32([nf])
    ncl, nn = (cl, n) if in_place else (torch.full_like(cl, 77), torch.full_like(n, 77))
    kw = {} if in_place else dict(new_context_lens=ncl, new_num_free=nn)
    pa.paged_blocks_release(bt, cl, torch.from_numpy(np.asarray(fin, bool)).to(dev()), fr, n, bs, num_blocks=NB, **kw)
    for g, w in zip((ncl, fr, nn), want):
        assert np.array_equal(g.cpu().numpy(), np.atleast_1d(w))
    assert pa.get_device_error() == bits(pa, want[3])
    assert np.array_equal(bt.cpu().numpy(), table)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,ctx,bs", [(1, 1, 16), (64, 4096, 16), (7, 100, 1), (300, 9000, 32), (5000, 20, 2), (16384, 9, 4)])
def test_release(pa, B, ctx, bs, in_place):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, ctx + 1, B).astype(np.int32)
    table, free, NB = pool(rng, lens, -(-ctx // bs), bs, 11)
    run_release(pa, table, lens, rng.random(B) < 0.4, free, 11, bs, NB, in_place)
    run_release(pa, table, lens, np.ones(B), free, 11, bs, NB, in_place)
    run_release(pa, table, lens, np.zeros(B), free, 11, bs, NB, in_place)


def test_release_out_of_range(pa):
    """Lengths out of range, a stack without room, a height out of range, bad ids."""
    rng = np.random.default_rng(4)
    lens = np.array([5, -1, 33, 7, 0, 12, 9], np.int32)
    table, free, NB = pool(rng, [5, 0, 32, 7, 0, 12, 9], 4, 8, 3)
    table[3, 0] = -5
    for cap in (3, 4, 5, 6, 8, len(free)):
        run_release(pa, table, lens, [1, 1, 1, 1, 1, 1, 0], free[:cap].copy(), 3, 8, NB)
    run_release(pa, table, lens, [1] * 7, free, -2, 8, NB)
    run_release(pa, table, lens, [1] * 7, free, len(free) + 9, 8, NB)
    run_release(pa, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), [], free, 3, 8, NB)


@pytest.mark.parametrize("plain", [False, True])
def test_release_onto_a_stack_shorter_than_the_pool(pa, monkeypatch, plain):
    """Without num_blocks every id goes back, whatever the stack's capacity."""
    if plain:
        monkeypatch.setattr(pa, "_binding", None)
    table, lens, free, n = t32([[900, 3], [77, 5000]]), t32([20, 9]), t32([8, 0, 0, 0]), t32([1])
    pa.paged_blocks_release(table, lens, torch.tensor([True, True], device=dev()), free, n, 16)
    assert free.tolist() == [8, 900, 3, 77] and int(n) == 4 and lens.tolist() == [0, 0]
    assert pa.get_device_error() == 0


def test_python_refusals(pa):
    bt, x2, x3, x8, one = (t32(np.zeros(s)) for s in ((2, 4), 2, 3, 8, 1))
    ok = [bt, x2, x2.clone(), x8, one, x3, x8.clone(), x8.clone(), 16, 8]
    pa.paged_blocks_append(*ok)
    for i, bad, exc in ((0, bt[0], ValueError), (0, bt.long(), TypeError), (1, x3, ValueError), (2, x3, ValueError), (2, x2.float(), TypeError),
                        (3, bt, ValueError), (4, x2, ValueError), (5, x2, ValueError), (6, bt, ValueError), (7, x3, ValueError),
                        (0, bt.t(), ValueError)):
        args = list(ok)
        args[i] = bad
        with pytest.raises(exc):
            pa.paged_blocks_append(*args)
    with pytest.raises(ValueError):
        pa.paged_blocks_append(*ok, new_context_lens=x3)
    with pytest.raises(pa.PagedAttnError):
        pa.paged_blocks_append(*ok[:8], 12, 8)
    with pytest.raises(TypeError):
        pa.paged_blocks_release(bt, x2, x2, x8, one, 16)
    with pytest.raises(ValueError):
        pa.paged_blocks_release(bt, x2, x3.bool(), x8, one, 16)
    assert pa.get_device_error() == 0
