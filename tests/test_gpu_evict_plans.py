"""Eviction's launch plans, bit for bit: the selection by one CTA, by clusters of 2, 4 and 8 and by
the kernel for longer rows, at the widths where one gives way to the next; rows moved whole and in
parts; what bad block ids leave alone."""
import numpy as np
import pytest
import torch

import compress_cases as cc
from gpu_cases import dev, pa_mod
from test_gpu_evict import back, caches, masses, on_gpu, reference, run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


# tokens that tables and masses hold: the last of one plan and the first of the next
WIDTHS = [16384, 16385, 32768, 32769, 65536, 65537, 131071, 393216, 393217]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["plain", "ties", "crowd", "special"])
def test_selection_plans(pa, width, kind, in_place):
    """A row of the whole width, next to rows that end in the first CTA's slice, hold one token or none."""
    lens = [width, 700, 0, 1, width // 3]
    keep = [width // 5, 300, 4, 1, width // 3 - 1]
    run_case(pa, width + len(kind), lens, keep, 37, 1, 64, 256, "int4", kind=kind, in_place=in_place, extra=0)


@pytest.mark.parametrize("width", [20000, 100000])
@pytest.mark.parametrize("keep,recent", [(1, 0), (19999, 0), (5000, 5000), (5000, 4999)])
def test_selection_of_nearly_all_and_nearly_none(pa, width, keep, recent):
    run_case(pa, 5, [width, 20000], [keep, keep], recent, 2, 64, 64, "bf16", kind="special", in_place=True, extra=0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,D", [("f32", 128), ("f32", 64), ("bf16", 128), ("bf16", 96), ("e4m3", 128), ("int4", 128),
                                     ("f32", 4096)])
@pytest.mark.parametrize("B", [1, 9])
def test_rows_moved_in_parts(pa, B, dtype, D, in_place):
    """Few rows, whose vectors are parted among clusters, and more of them."""
    rng = np.random.default_rng(B + D)
    lens = rng.integers(300, 900, B)
    run_case(pa, 7 + D, lens, lens // 2, 5, 1, D, 16, dtype, in_place=in_place)


@pytest.mark.parametrize("dtype", ["bf16", "int4"])
@pytest.mark.parametrize("side", ["source", "destination"])
def test_rows_of_bad_blocks_stay(pa, dtype, side):
    """Bad ids in one of the tables: their rows are not moved, every other row is, indices and masses are
    those of good tables, and the error is reported."""
    d = dev()
    rng = np.random.default_rng(35)
    Hk, D, bs, n, keep = 2, 64, 16, 64, 40
    bt = np.arange(12, dtype=np.int32).reshape(3, 4)
    obt = np.arange(12, 21, dtype=np.int32).reshape(3, 3)
    arrays = caches(rng, 21, bs, Hk, D, dtype)
    mass = masses(rng, (3, Hk, n), "plain")
    lens, keeps = np.full(3, n, np.int32), np.full(3, keep, np.int32)
    kept, mo, _ = reference(None, mass, lens, keeps, 2, bt, obt, bs, keep, keep, arrays, dtype == "int4")
    bad = (bt if side == "source" else obt).copy()
    bad[1, 1], bad[2, 0], bad[0, 2] = 21, -1, 1 << 30
    tables = (bad, obt) if side == "source" else (bt, bad)
    want = [None if a is None else a.copy() for a in arrays]
    for b in range(3):
        for h in range(Hk):
            for i in range(keep):
                s, t = kept[b, h, i], i
                sb, db = tables[0][b, s // bs], tables[1][b, t // bs]
                if not (0 <= sb < 21 and 0 <= db < 21):
                    continue
                for w, a in zip(want, arrays):
                    if a is not None:
                        if dtype == "int4":
                            w[db, h, t % bs] = a[sb, h, s % bs]
                        else:
                            w[db, t % bs, h] = a[sb, s % bs, h]
    assert any(not np.array_equal(w.view(np.uint8), a.view(np.uint8)) for w, a in zip(want, arrays) if a is not None)
    t = [on_gpu(a, dtype if i < 2 else "int4") for i, a in enumerate(arrays)]
    kd, mod = torch.empty((3, Hk, keep), dtype=torch.int32, device=d), torch.empty((3, Hk, keep), device=d)
    pa.paged_kv_evict(kd, torch.from_numpy(mass).to(d), mod, t[0], t[1], *(torch.from_numpy(x).to(d) for x in tables),
                      torch.from_numpy(lens).to(d), torch.from_numpy(keeps).to(d), 2, kv_params=t[2])
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(kd.cpu().numpy(), kept) and np.array_equal(mod.cpu().numpy(), mo)
    for got, w in zip(t, want):
        if w is not None:
            assert np.array_equal(back(got, w).view(np.uint8), w.view(np.uint8))
