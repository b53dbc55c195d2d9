"""Every way that the block-scaled decode can go, for both head sizes: clusters of one to sixteen CTAs that take a
row, runs of stages whose partials 1, 4 or 32 warps join. Which way a call went is read off its launches."""
import numpy as np
import pytest
import torch

from gpu_cases import dev, pa_mod
from launches import launches
from test_gpu_fp8_block import RUNS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def way(pa, case, bound):
    """("rows", CTAs of a cluster) or ("runs", warps that join a row) of a call, and its padded group."""
    t, out = case.t, torch.empty_like(case.t["q"])
    B, MB = case.bt.shape
    ws = torch.empty(pa.decode_fp8_block_workspace_bytes(B, case.H, case.Hk, case.D, bound or MB * case.bs), dtype=torch.uint8,
                     device=dev())
    got = launches(lambda: case.run(pa, out=out, max_context_len=bound, workspace=ws))
    heads = 8 if case.H // case.Hk <= 8 else 16
    rows = B * case.Hk
    main = f"Li{case.D}ELi{heads}ELb"
    if len(got) == 1:
        cluster = got[0].cluster[0]
        assert main + "1E" in got[0].name and got[0].grid == (rows * cluster, 1, 1)
        return "rows", cluster
    assert len(got) == 2 and main + "0E" in got[0].name and "decode_join_kernel" in got[1].name
    joins = [w for w in (1, 4, 32) if f"Li{case.D}ELi{w}E" in got[1].name]
    assert len(joins) == 1
    return "runs", joins[0]


# Lengths in stages (64 tokens of 64 channels, 32 of 128), less the tokens given, so that the last stage is a part;
# H, Hk; the bound in stages, or None for one at which any call is cut into runs; what 152 SMs are expected to make of it.
WAYS = [
    ([(1, 3), (0, 0), (8, 1)], 8, 2, 8, ("rows", 1)), ([(7, 0)] * 18, 32, 8, 8, ("rows", 1)),
    ([(16, 5), (1, 1), (9, 0)], 12, 3, 16, ("rows", 2)), ([(16, 0), (2, 7)], 16, 1, 16, ("rows", 2)),
    ([(32, 31), (20, 0), (1, 0)], 6, 2, 32, ("rows", 4)), ([(30, 0), (17, 9), (0, 0)], 24, 2, 32, ("rows", 4)),
    ([(64, 1), (33, 0), (2, 2)], 4, 2, 64, ("rows", 8)), ([(50, 9), (64, 0)], 28, 2, 64, ("rows", 8)),
    ([(141, 24), (70, 0)], 8, 2, 141, ("rows", 16)), ([(141, 24)], 9, 1, 141, ("rows", 16)), ([(256, 0)], 4, 1, 256, ("rows", 16)),
    ([(141, 24)], 8, 1, None, ("runs", 32)), ([(200, 3), (1, 0)], 20, 2, None, ("runs", 32)), ([(34, 1)], 16, 1, None, ("runs", 32)),
    ([(60, 1), (3, 0), (33, 9)] * 14, 8, 1, None, ("runs", 4)), ([(90, 0)] + [(4, 1)] * 41, 16, 1, None, ("runs", 4)),
    ([(9, 4), (40, 0), (0, 0), (1, 2)] * 10, 32, 4, None, ("runs", 1)), ([(9, 4), (40, 0)] * 80, 12, 1, None, ("runs", 1))]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (64, 128)])
@pytest.mark.parametrize("lens,H,Hk,bound,expected", WAYS)
def test_every_way(pa, lens, H, Hk, bound, expected, D, bs, dtype):
    tok = 4096 // D
    case = Case(np.random.default_rng(81 + H + D), [s * tok - less for s, less in lens], H, Hk, D, bs, dtype, gain=2.0)
    bound = RUNS if bound is None else bound * tok
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert way(pa, case, bound) == expected
    out = case.run(pa, max_context_len=bound)
    case.check(out)
    assert torch.equal(out, case.run(pa, max_context_len=bound)) and pa.get_device_error() == 0
