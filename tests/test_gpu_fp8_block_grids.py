"""The grids of the block-scaled scatter and read-back: what the device holds, for every type."""
import pytest
import torch

from gpu_cases import dev, pa_mod
from launches import launches

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def cache(NB, Hk, bs, D):
    kc = torch.zeros((NB, Hk, bs, D), dtype=torch.uint8, device=dev())
    return kc, torch.zeros_like(kc), torch.ones((NB, Hk, 2), device=dev())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,Hk,D,bs", [(1, 8, 128, 16), (64, 8, 128, 16), (1000, 8, 128, 16), (2048, 8, 128, 16), (2000, 4, 64, 16),
                                       (700, 2, 128, 64), (300, 5, 64, 8)])
def test_scatter_of_few_columns_fills_the_device_once(pa, dtype, T, Hk, D, bs):
    """Few columns of 32 tokens aim at as many CTAs as the device holds at once, and no more."""
    c = cache(8, Hk, bs, D)
    k = torch.zeros((T, Hk, D), dtype=dtype, device=dev())
    slots = torch.full((T,), -1, dtype=torch.int32, device=dev())
    (w,) = launches(lambda: pa.paged_kv_write_fp8_block(k, k, slots, *c))
    columns, room = -(-T // 32), sms() * w.held
    assert "kv_write_fp8_block" in w.name and w.grid[0] % columns == 0
    assert w.grid[0] <= room
    # a warp for each step of single tokens, or no room for another CTA of every column
    singles = -(-32 * -(-2 * Hk // (32 // (D // 16))) // 4)
    assert w.grid[0] // columns == singles or w.grid[0] + columns > room
