"""4-bit decode over bad block ids: their tokens count with score and value 0, within the bound of
the decode tests."""
import numpy as np
import pytest
import torch

from gpu_cases import dev, pa_mod
from test_gpu_int4 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return pa_mod()


@pytest.mark.parametrize("H,Hk,D,bs,bad", [(8, 2, 128, 16, (2, 5)), (12, 1, 64, 8, (0, 12)), (8, 2, 128, 128, (0,))])
def test_bad_blocks_read_as_zeros(pa, H, Hk, D, bs, bad):
    """Some blocks of one sequence, its last and partly filled one among them; then every one."""
    n = 100
    case = Case(np.random.default_rng(71), [n, 60], H, Hk, D, bs, "bf16")
    want = case.run(pa)[1].clone()
    for j, blocks in enumerate((bad, range(-(-n // bs)))):
        for i in blocks:
            b = case.bt[0, i]
            case.t["bt"][0, i] = (case.NB, -1, 1 << 30)[(i + j) % 3]
            case.kc[b], case.vc[b], case.par[b] = 0, 0, 0
            case.k[0][i * bs:(i + 1) * bs], case.v[0][i * bs:(i + 1) * bs] = 0.0, 0.0
        mass = torch.zeros((2, Hk, n), device=dev())
        out = case.run(pa, mass)
        assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_ID
        case.check(out, mass)
        assert torch.equal(out[1], want)
    assert (out[0] == 0).all()
