"""The operators around a stack's blocks at values that their formulas allow and few inputs hold. Tolerances as
in test_gpu_stack."""
import numpy as np
import pytest
import torch

from test_gpu_stack import BF, DEV, F32, F64, U, check_norm_grad, gen, norm_grad_ref, randn, within, words

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


# Row lengths that fill the last round of a row's chunks and ones that do not; rows that fill the last unit of
# rows and ones that do not.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 72), (37, 264), (1531, 264), (700, 2056), (9, 4096), (701, 4104), (1301, 7168),
                                 (2, 8200)])
def test_gradient_of_rows_of_one_huge_value(M, T, H, dtype):
    """x - mean is 0 in such a row, and so is all that is multiplied by it, though mean * rstd is over the
    largest number (2^120 * 2^10)."""
    g = gen(T + H)
    x, dh, dres = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype)
    gamma, beta = 1 + randn(g, H, std=0.3), randn(g, H)
    eps = 2.0 ** -20
    n = M.layer_norm(x, gamma, beta, eps)
    huge = torch.arange(T, device=DEV) % 3 == 0  # the first row among them
    x[huge] = 2.0 ** 120
    n.mean[huge] = 2.0 ** 120
    n.rstd[huge] = 2.0 ** 10
    for res in (dres, None):
        got = M.layer_norm_backward(dh, x, gamma, n.mean, n.rstd, dres=res)
        check_norm_grad(got.dx, got.dgamma, got.dbeta, dh, x, gamma, n.mean, n.rstd, res, True)
        rng = torch.tensor([3, 4], device=DEV)
        b = M.dropout_join_backward(res, 0.25, rng, 1, 1.0, dh, x, gamma, n.mean, n.rstd)
        check_norm_grad(b.dx, b.dgamma_next, b.dbeta_next, dh, x, gamma, n.mean, n.rstd, res, True)
        f = torch.from_numpy((words(T * H, 3, 4, 1) >= np.uint64(1 << 30)).reshape(T, H)).to(DEV).to(F64) / 0.75
        dx, off, _ = norm_grad_ref(dh, x, gamma, n.mean, n.rstd, res)
        within(b.dy, f * dx, f * (off + 3 * U * dx.abs()), "dy")


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


def test_probabilities_of_sigmoids_far_below_the_largest(M):
    """A sequence a token: prob is the tokens' probabilities. A sigmoid of z < 0 is x / (1 + x), x = exp(z): off by 2
    steps (an exponential, whatever its argument), a step for the reciprocal, and half a step for 1 + x and the
    product: 8 half steps. The sum over experts is off by as much and half a step for each of 16 + 5
    additions, its reciprocal and the last product by one each: 39."""
    g = gen(31)
    T, E, k = 700, 64, 2
    z = -80 * torch.rand(T, E, generator=g, device=DEV)
    z[:, ::16] = randn(g, T, 4).abs()
    ids = z.topk(k, 1).indices.to(torch.int32)
    offsets = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    b = M.balance_loss(z, ids, mode=1, offsets=offsets)
    ref = torch.sigmoid(z.to(F64))
    ref = ref / ref.sum(1, keepdim=True)
    assert (b.prob.to(F64) / ref - 1).abs().max() <= 40 * U


def test_dropout_on_both_sides_of_the_2_34th_element(M, L):
    """From there on the upper word of the generator's counter is not 0. In place, through the C entry point."""
    H = 32768
    T = (1 << 34) // H + 3
    if torch.cuda.mem_get_info()[0] < 3 * T * H:
        pytest.skip("not enough free memory")
    x = torch.ones(T, H, dtype=BF, device=DEV)
    rng = torch.tensor([2 ** 62 + 77, 2 ** 35 + 1], device=DEV)
    cfg = L.moe_layer_t(T=T, H=H, dtype=L.MOE_BF16, scale=1.0)
    L.moe_dropout(cfg, L.moe_drop_t(p=0.5, rng=rng.data_ptr(), site=9), x, x)
    start = (T - 6) * H
    want = torch.from_numpy(words(6 * H, 2 ** 62 + 77, 2 ** 35 + 1, 9, start) >= np.uint64(1 << 31)).view(6, H)
    assert start < 1 << 34 < T * H
    assert torch.equal(x[-6:].cpu(), 2.0 * want.to(BF))
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1215, 1024), (1217, 1024), (2433, 1024), (3, 1032), (700, 1032), (2433, 1032), (307, 2304),
                                 (152, 2312), (153, 2312), (457, 2312), (155, 4096)])
def test_norm_gradient_around_its_kernels_borders(M, T, H, dtype):
    """One or two chunks a thread go by the length of a row and the number of rows."""
    g = gen(T * 3 + H)
    x, dh, dres = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype)
    gamma, beta = 1 + randn(g, H, std=0.3), randn(g, H)
    n = M.layer_norm(x, gamma, beta)
    got = M.layer_norm_backward(dh, x, gamma, n.mean, n.rstd, dres=dres)
    check_norm_grad(got.dx, got.dgamma, got.dbeta, dh, x, gamma, n.mean, n.rstd, dres, True)
    assert all(torch.equal(a, b) for a, b in zip(got, M.layer_norm_backward(dh, x, gamma, n.mean, n.rstd, dres=dres)))
