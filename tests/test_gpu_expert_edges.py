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


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("renormalise", [True, False])
def test_a_softmax_of_nan_or_infinity_shows_in_every_weight(lib, bad, renormalise):
    """Also where the choice leaves the bad logit out: with a bias, or worths of two keys, every key
    of the token is NaN and the lowest experts come first.  The other tokens see nothing of it."""
    x = torch.randn(40, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    x[1::4, 37] = bad
    x[1::4, 5] = -float("inf")
    bias = torch.zeros(64, device="cuda")
    for b, kw in ((bias, {}), (bias, dict(groups=4, top_groups=2)),
                  (bias, dict(groups=4, top_groups=2, group_keys=2)),
                  (None, dict(groups=4, top_groups=2, group_keys=2)),
                  (None, dict(groups=4, top_groups=2)), (None, {})):
        idx, w = routes.forward(lib, x, b, 6, score="softmax", renormalise=renormalise, **kw)
        assert (idx >= 0).all() and not (idx[1::4] == 5).any()
        assert torch.isnan(w[1::4]).all(), kw
        for k in (0, 2, 3):
            assert torch.isfinite(w[k::4]).all(), kw
    # slots that no expert is left for keep weight 0
    x[1::4] = -float("inf")
    x[1::4, 37:39] = bad
    idx, w = routes.forward(lib, x, bias, 6, score="softmax", renormalise=renormalise)
    assert (idx[1::4] >= 0).sum(1).eq(2).all()
    assert torch.equal(torch.isnan(w[1::4]), idx[1::4] >= 0) and (w[1::4, 2:] == 0).all()
