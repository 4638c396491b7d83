"""Gradients of routing and rows where a program asks for less than all of them, or hands over tensors that are not its own."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()


def _rand(*shape, seed=0):
    import torch
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_options_are_the_forward_calls():
    """An option given as a tensor that changes afterwards: the gradient is that of the forward call."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    G = _rand(20, 3, seed=4)

    def grad(change):
        logits = _rand(20, 8, seed=1).requires_grad_()
        scale, renormalize = torch.tensor(2.0), torch.tensor(True)
        w = ag.route(logits, 3, scale=scale, renormalize=renormalize).weight
        if change:
            scale.fill_(5.0)
            renormalize.fill_(False)
        w.backward(G)
        return logits.grad

    assert torch.equal(grad(True), grad(False))
