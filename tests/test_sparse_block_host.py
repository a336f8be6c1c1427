"""What a trainable block refuses, by name, before anything is enqueued: its router reaches the library
by address, so a tensor of another type, layout or device would be misread, not refused there."""
import pytest
import torch

BF, F32 = torch.bfloat16, torch.float32
E, H, I = 4, 64, 48


@pytest.fixture(scope="module")
def S():
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import sparse_block
    return sparse_block


def parameters(dtype=BF, **kw):
    p = dict(Wg=torch.zeros(E, H, dtype=dtype), W13=torch.zeros(E, 2 * I, H, dtype=dtype),
             W2=torch.zeros(E, H, I, dtype=dtype), gamma_in=torch.ones(H), gamma_out=torch.ones(H), k=2)
    return {**p, **kw}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_matching_parameters_are_taken(S, dtype):
    S.SparseBlock(**parameters(dtype))
    S.SparseBlock(**parameters(dtype, gate=torch.ones(H), logit_bias=torch.zeros(E), select_bias=torch.zeros(E)))
    for gate in (torch.ones(7, 1), torch.ones(7, H, dtype=dtype)):  # one a token, one an element
        S.SparseBlock(**parameters(dtype, gate=gate))


WRONG = [
    # a router kept in fp32 beside bf16 experts, and the reverse
    (dict(Wg=torch.zeros(E, H)), "W13: dtype"),
    (dict(W2=torch.zeros(E, H, I)), "W2: dtype"),
    (dict(Wg=torch.zeros(E, H, dtype=torch.float16)), "Wg"),
    (dict(Wg=torch.zeros(H, E, dtype=BF).T), "Wg: has to be contiguous"),
    (dict(Wg=torch.zeros(E * H, dtype=BF)), "Wg"),
    (dict(Wg=[[0.0] * H] * E), "Wg"),
    (dict(Wg=torch.zeros(E, H, dtype=BF, device="meta")), "W13: is on cpu"),
    (dict(W13=torch.zeros(E, H, 2 * I, dtype=BF).transpose(1, 2)), "W13: has to be contiguous"),
    (dict(W2=torch.zeros(E, H, I, dtype=BF, device="meta")), "W2: is on meta"),
    (dict(logit_bias=torch.zeros(E, dtype=BF)), "logit_bias: dtype"),
    (dict(select_bias=torch.zeros(E, dtype=BF)), "select_bias: dtype"),
    (dict(logit_bias=torch.zeros(E + 1)), "logit_bias: shape"),
    (dict(select_bias=torch.zeros(2 * E)[::2]), "select_bias: has to be contiguous"),
    (dict(logit_bias=torch.zeros(E, device="meta")), "logit_bias: is on meta"),
    (dict(gamma_in=torch.ones(H, dtype=BF)), "gamma_in: dtype"),
    (dict(gamma_out=torch.ones(H + 8)), "gamma_out: shape"),
    (dict(gamma_out=None), "gamma_out: a tensor is needed"),
    (dict(gate=torch.ones(H, device="meta")), "gate: is on meta"),
    (dict(gate=torch.ones(H, dtype=BF)), "gate: dtype"),
    (dict(gate=torch.ones(3, H)), "gate: dtype"),
    (dict(gate=torch.ones(3, 1, 1)), "gate: shape"),
    (dict(gate=torch.ones(H + 1)), "gate: shape"),
    (dict(gate=0.5), "gate: a tensor is needed"),
]


@pytest.mark.parametrize("kw,said", WRONG)
def test_parameters_that_would_be_misread_are_refused(S, kw, said):
    with pytest.raises(ValueError, match=said):
        S.SparseBlock(**parameters(**kw))


@pytest.mark.parametrize("name,wrong,said", [
    ("Wg", torch.zeros(E, H), "Wg: dtype"), ("Wg", torch.zeros(E, 2 * H, dtype=BF)[:, ::2], "Wg: has to be contiguous"),
    ("logit_bias", torch.zeros(E, dtype=BF), "logit_bias: dtype"),
    ("select_bias", torch.zeros(E - 1), "select_bias: shape")])
def test_parameters_replaced_later_are_checked_by_the_call(S, name, wrong, said):
    b = S.SparseBlock(**parameters())
    setattr(b, name, wrong)
    with pytest.raises(ValueError, match=said):
        b.route(torch.zeros(3, H, dtype=BF))


@pytest.mark.parametrize("x,said", [
    (torch.zeros(3, H), "dtype"), (torch.zeros(3, H + 8, dtype=BF), "shape"), (torch.zeros(H, dtype=BF), "shape"),
    (torch.zeros(3, 2 * H, dtype=BF)[:, ::2], "has to be contiguous"),
    (torch.zeros(3, H, dtype=BF, device="meta"), "is on meta"),
    (torch.zeros(3, H, dtype=BF), "has to be on the current CUDA device"), (None, "a tensor is needed")])
def test_tokens_that_do_not_fit_are_refused(S, x, said):
    b = S.SparseBlock(**parameters())
    with pytest.raises(ValueError, match="h: .*" + said):
        b.route(x)
    with pytest.raises(ValueError, match="x: .*" + said):
        S.SparseStack([b]).forward(x)


def test_blocks_of_a_stack_share_their_tokens_type_and_width(S):
    b = S.SparseBlock(**parameters())
    with pytest.raises(ValueError, match=r"blocks\[1\].Wg: dtype"):
        S.SparseStack([b, S.SparseBlock(**parameters(F32))])
    narrow = parameters(Wg=torch.zeros(E, 32, dtype=BF), W13=torch.zeros(E, 2 * I, 32, dtype=BF),
                        W2=torch.zeros(E, 32, I, dtype=BF), gamma_in=torch.ones(32), gamma_out=torch.ones(32))
    with pytest.raises(ValueError, match=r"blocks\[1\].Wg: shape"):
        S.SparseStack([b, S.SparseBlock(**narrow)])
