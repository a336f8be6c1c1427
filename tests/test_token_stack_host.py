"""What the stack that trains from token ids refuses, by name, without a GPU."""
import pytest
import torch

BF = torch.bfloat16
E, H, I, V = 4, 64, 48, 20


@pytest.fixture(scope="module")
def S():
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import token_stack
    return token_stack


def block(S, dtype=BF, h=H, **kw):
    p = dict(Wg=torch.zeros(E, h, dtype=dtype), W13=torch.zeros(E, 2 * I, h, dtype=dtype),
             W2=torch.zeros(E, h, I, dtype=dtype), gamma=torch.ones(h), beta=torch.zeros(h), k=2)
    return S.TokenBlock(**{**p, **kw})


@pytest.mark.parametrize("kw,said", [
    (dict(gamma=torch.ones(H + 8)), "gamma: shape"), (dict(gamma=torch.ones(H, dtype=BF)), "gamma: dtype"),
    (dict(beta=torch.ones(H, 1)), "beta: shape"), (dict(beta=torch.ones(2 * H)[::2]), "beta: has to be contiguous"),
    (dict(W13=torch.zeros(E, 2 * I, H)), "W13: dtype"), (dict(logit_bias=torch.zeros(E + 1)), "logit_bias: shape"),
    (dict(gamma=None), "gamma: a tensor")])
def test_block_refuses(S, kw, said):
    with pytest.raises(ValueError, match=f"^{said}"):
        block(S, **kw)


@pytest.mark.parametrize("kw,said", [
    (dict(blocks=[]), "blocks: at least one"), (dict(p=1.0), "p: 1.0"), (dict(p=-0.5), "p: -0.5"),
    (dict(table=torch.zeros(V, H)), "table: dtype"), (dict(table=torch.zeros(V, H + 8, dtype=BF)), "table: shape"),
    (dict(gamma_final=torch.ones(H, dtype=BF)), "gamma_final: dtype"),
    (dict(beta_final=torch.ones(H + 1)), "beta_final: shape")])
def test_stack_refuses(S, kw, said):
    a = dict(table=torch.zeros(V, H, dtype=BF), blocks=[block(S), block(S, beta=None)], gamma_final=torch.ones(H)) | kw
    with pytest.raises(ValueError, match=f"^{said}"):
        S.TokenStack(**a)


def test_stack_refuses_blocks_that_do_not_fit(S):
    with pytest.raises(ValueError, match=r"^blocks\[1\].Wg: dtype"):
        S.TokenStack(torch.zeros(V, H, dtype=BF), [block(S), block(S, dtype=torch.float32)], torch.ones(H))
    with pytest.raises(ValueError, match=r"^blocks\[1\].Wg: shape"):
        S.TokenStack(torch.zeros(V, H, dtype=BF), [block(S), block(S, h=H + 8)], torch.ones(H))


def test_parameters_and_gradients(S):
    s = S.TokenStack(torch.zeros(V, H, dtype=BF), [block(S), block(S, beta=None)], torch.ones(H), seed=5)
    assert set(s.parameters()) == set(s.grads) == {"table", "gamma_final"}
    assert [set(g) for g in s.block_grads] == [{"Wg", "W13", "W2", "gamma", "beta"}, {"Wg", "W13", "W2", "gamma"}]
    assert all(t.dtype == torch.float32 for g in [s.grads, *s.block_grads] for t in g.values())
    assert s.rng.tolist() == [5, 0]
