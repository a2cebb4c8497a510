"""Calls of the routed layer whose work is more than one launch takes (2^32 threads): every row right, on both sides
of the launches' borders.  Inputs are whole numbers that bf16 holds, so results are exact."""

import pytest
import torch

from expert_ffn_ragged_amd import rd
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def small_whole(shape):
    """Values -4 .. 3 that depend on the place."""
    n = 1
    for s in shape:
        n *= s
    return ((torch.arange(n, device=DEV, dtype=torch.int32) * 2654435 >> 9) % 8 - 4).to(torch.bfloat16).view(shape)


def test_dispatch_and_combine_gradients_of_67_million_choices():
    tokens, top_k, hidden = (1 << 23) + 3, 8, 8
    say(f"dispatch_rows and combine_rows_bwd {tokens} x {top_k}")
    n = tokens * top_k
    slots = (n - 1 - torch.arange(n, device=DEV, dtype=torch.int32)).view(tokens, top_k)
    x = small_whole((tokens, hidden))
    xs = rd.dispatch_rows(x, slots)
    assert torch.equal(xs.flip(0).view(tokens, top_k, hidden), x[:, None].expand(-1, top_k, -1))
    weights = torch.full((tokens, top_k), 2.0, device=DEV)
    dy, dw = rd.combine_rows_bwd(x, xs, slots, weights)
    assert torch.equal(dy, xs + xs)
    assert torch.equal(dw, x.float().square().sum(1, keepdim=True).expand(-1, top_k))


def test_combine_of_67_million_tokens():
    tokens, hidden = (1 << 26) + 5, 8
    say(f"combine_rows {tokens}")
    slots = (tokens - 1 - torch.arange(tokens, device=DEV, dtype=torch.int32)).view(tokens, 1)
    y = small_whole((tokens, hidden))
    assert torch.equal(rd.combine_rows(y, slots), y.flip(0))


@pytest.mark.parametrize("experts,tokens", [(2, (1 << 28) + 7), (257, (1 << 26) + 7)])
def test_route_and_gradient_of_many_tokens(experts, tokens):
    say(f"route {tokens} x {experts}")
    logits = torch.zeros((tokens, experts), dtype=torch.bfloat16, device=DEV)
    best = torch.arange(tokens, device=DEV) * 7919 % experts
    logits.scatter_(1, best[:, None], 1.0)
    w, ids = rd.route(logits, 1)
    assert bool((ids[:, 0] == best).all())
    assert bool((w == w[0]).all()) and abs(w[0].item() * (1 + (experts - 1) / 2.718281828459045) - 1) < 1e-6
    if experts > 2:  # the gradient of the small one: the other kernels differ in the lanes of a row alone
        return
    grad = rd.route_bwd(logits, ids, torch.ones_like(w))
    p = w[0].item()
    mine = grad.gather(1, best[:, None])
    other = grad.gather(1, 1 - best[:, None])
    assert bool((mine == mine[0]).all()) and bool((other == -mine[0]).all())
    assert abs(mine[0].item() - p * (1 - p)) <= 2.0 ** -8 * p * (1 - p)
