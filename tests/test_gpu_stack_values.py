"""The operators around a stack's blocks at values that their formulas allow and few inputs hold. Tolerances as
in test_gpu_stack."""
import pytest
import torch

from test_gpu_stack import BF, DEV, F32, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import _lib
    _lib.moe_device_status(True)
    return _lib


@pytest.fixture(scope="module")
def M(L):
    from routing_grouped_gemm_router_gb300 import training
    return training


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(3, 72), (700, 2056), (700, 4096), (37, 16384)])
def test_the_join_adds_what_dropout_gives(M, T, H, dtype):
    """out is x + dropout(y) with the bits of dropout in fp32 and one more addition: bf16 rows times 1 / 0.9 lie so
    often next to the middle of two bf16 values that another rounding on the way is seen in one of 2000."""
    g = gen(T + H)
    x, y = randn(g, T, H, dtype=dtype, std=1.6), randn(g, T, H, dtype=dtype)
    gamma, rng = 1 + randn(g, H, std=0.2), torch.tensor([21, 5], device=DEV)
    for p, scale in ((0.1, 1.0), (0.1, 0.7), (0.5, 1.0), (0.0, 0.5)):
        want = (x.float() + M.dropout(y.float(), p, rng, 4, scale)).to(dtype)
        assert torch.equal(M.dropout_join(x, y, p, rng, 4, scale).out, want)
        assert torch.equal(M.dropout_join(x, y, p, rng, 4, scale, gamma).out, want)
