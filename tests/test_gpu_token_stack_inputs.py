"""The stack that trains from token ids: what a program may change between a forward and its backward pass."""
import pytest
import torch

from test_gpu_token_stack import DEV, H, S, make, tokens_of  # noqa: F401

pytestmark = pytest.mark.gpu


def test_inputs_may_be_written_before_the_backward_pass(S):
    """A program that fills its buffers with the next batch before it runs backward gets the gradients of the
    batch that it ran forward."""
    T = 64
    stack, rnd = make(S, torch.float32, p=0.2)
    dh, up = rnd(T, H), torch.tensor([0.3, 0.05], device=DEV)
    tokens = tokens_of(T, 5)
    offsets = torch.tensor([0, 20, 30, 60], dtype=torch.int32, device=DEV)
    mask = torch.arange(T, device=DEV) % 5 != 0

    def grads(between):
        stack.zero_grad()
        saved = stack.forward(tokens, offsets, mask)[2]
        between()
        stack.backward(dh, saved, up)
        return [t.clone() for g in (stack.grads, *stack.block_grads) for t in g.values()]

    def next_batch():
        tokens.copy_(tokens_of(T, 6))
        offsets.copy_(torch.tensor([0, 5, 50, 64]))
        mask.logical_not_()

    want = grads(lambda: None)
    got = grads(next_batch)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_pass_without_dropout_between_forward_and_backward(S):
    """A validation pass with p set to 0 in between leaves the gradients as they are."""
    T = 40
    stack, rnd = make(S, torch.float32, p=0.3)
    tokens, dh = tokens_of(T, 5), rnd(T, H)

    def grads(between):
        stack.p = 0.3
        stack.zero_grad()
        saved = stack.forward(tokens)[2]
        between()
        stack.backward(dh, saved)
        return [t.clone() for g in (stack.grads, *stack.block_grads) for t in g.values()]

    def validate():
        stack.p = 0.0
        stack.forward(tokens_of(T, 6))

    want = grads(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(grads(validate), want))
