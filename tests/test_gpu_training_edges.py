"""The training operators where their loops and warps take the less usual way: rows by the thousand
through the norms' rings, results that lanes of one warp store and others do not, sums next to the
ends of fp32's range. References in 64 bits; bounds are derived as in test_gpu_training."""
import pytest
import torch

from test_gpu_training import (DEV, DTYPES, F64, L, M, U, gen, randn, runs, within,  # noqa: F401
                               test_join_and_its_gradient as join_and_its_gradient)

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


# Results of M rows where M is no multiple of 32: some lanes of a warp hold rows to add to, others do not,
# while all of them load tensor memory together.
@pytest.mark.parametrize("Mm", [8, 40, 72, 136, 264, 392])
@pytest.mark.parametrize("N", [64, 136, 520])
def test_bf16_weight_gradients_added_to_by_part_of_a_warp(M, Mm, N):
    counts = [40, 0, 1, 130, 16]
    rs, P = runs(counts)
    g = gen(Mm + N)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    dy, a = randn(g, P, Mm, dtype=BF) * live, randn(g, P, N, dtype=BF) * live
    dW = randn(g, len(counts), Mm, N, dtype=BF)
    before = dW.clone()
    M.expert_weight_grad(dy, a, torch.tensor(counts, dtype=torch.int32, device=DEV), out=dW, accumulate=True)
    for e, r in rs:
        d, v = dy[r].to(F64), a[r].to(F64)
        mag = d.abs().T @ v.abs() + before[e].to(F64).abs()
        within(dW[e], before[e].to(F64) + d.T @ v, (r.stop - r.start + 3) * U * mag, BF, f"expert {e}")
