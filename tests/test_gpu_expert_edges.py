"""GPU: edges of routing by scores, of the quantiser and of the products on block-scaled fp8."""
import numpy as np
import pytest
import torch

from tests import test_gpu_route_scores as routes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,groups", [(16, 8), (64, 8), (96, 3)])
@pytest.mark.parametrize("size", [256.0, 1e4, 1e5, 1e6, 1e7])
def test_groups_whose_two_largest_keys_cancel(lib, E, groups, size):
    """One expert of a group with a bias of +size, the others -size: a worth is of the size of the
    scores, its rounding in 32 bits of the size of the keys that it is the sum of."""
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    x = torch.randn(65536, E, device="cuda", generator=g)
    bias = torch.full((groups, E // groups), -size, device="cuda")
    bias[torch.arange(groups), torch.arange(groups) % (E // groups)] = size
    for score in ("sigmoid", "softmax"):
        routes.check(lib, x, bias.view(-1), 4, score=score, groups=groups, top_groups=groups // 2 or 1,
                     group_keys=2)
