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


def codes_with_signs(x, bn, bk):
    """E4M3 codes by IEEE division on the CPU, zeros with x's sign, also under a scale of 0."""
    n, K = x.shape
    full = torch.zeros(-(-n // bn) * bn, -(-K // bk) * bk)
    full[:n, :K] = x.float()
    parts = full.view(full.shape[0] // bn, bn, full.shape[1] // bk, bk)
    s = (parts.abs().amax((1, 3)) / 448.0)[:, None, :, None]
    q = torch.where(s > 0, parts / s, torch.copysign(torch.zeros(()), parts)).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(full.shape)[:n, :K]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_codes_keep_the_sign_of_zero(lib, dtype):
    """Zeros of both signs, values that round to zero, blocks of nothing but zeros, and (fp32, bf16)
    blocks whose scale is outside the range of the corrected quotient, or zero: the same code
    whatever the form and whatever the blocks beside it."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn(300, 400, generator=g)
    x *= torch.exp2(torch.randint(-14, 2, (300, 400), generator=g).float())
    x = torch.where(torch.rand(300, 400, generator=g) < 0.3, torch.copysign(torch.zeros(()), x), x)
    x[:, 128:256] = torch.copysign(torch.zeros(300, 128), x[:, 128:256])
    x[128:256, 300:] = torch.copysign(torch.zeros(128, 100), x[128:256, 300:])
    if dtype != torch.float16:
        x[:128, 17] *= 2.0 ** 100
        x[200] *= 2.0 ** -100
    if dtype == torch.float32:
        x[256:, 260] = torch.copysign(torch.full((44,), 2.0 ** -147), x[256:, 260])
        x[10, :128] = torch.copysign(torch.full((128,), 2.0 ** -147), x[10, :128])
    x = x.to(dtype)
    assert (x.view(torch.int16 if dtype != torch.float32 else torch.int32) < 0)[x == 0].any()
    new = dict(dtype=torch.uint8, device="cuda")
    b = lib.fp8_blocks
    rc, cc, rc2, cc2, tc = (torch.empty(x.shape, **new) for _ in range(5))
    rs, cs = torch.empty(300, b(400), device="cuda"), torch.empty(b(300), 400, device="cuda")
    lib.moe_quantize_fp8(x.cuda(), rc, rs, cc, cs)
    lib.moe_quantize_fp8(x.cuda(), rc2, rs)
    lib.moe_quantize_fp8(x.cuda(), col_codes=cc2, col_scales=cs)
    lib.moe_quantize_fp8_tiles(x.cuda()[None], tc[None], torch.empty(1, b(300), b(400), device="cuda"))
    for got, block, name in ((rc, (1, 128), "rows of both"), (rc2, (1, 128), "rows"),
                             (cc, (128, 1), "columns of both"), (cc2, (128, 1), "columns"),
                             (tc, (128, 128), "tiles")):
        ref = codes_with_signs(x, *block)
        assert torch.equal(got.cpu(), ref), f"{name}: {(got.cpu() != ref).sum()} codes"


def test_zeros_of_rows_are_those_of_the_fp8_dispatch(lib):
    T, d, E = 130, 256, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, d, device="cuda", generator=g)
    x = torch.where(torch.rand(T, d, device="cuda", generator=g) < 0.5, x * 0.0, x).bfloat16()
    x[::3, :128] *= 0.0
    idx = torch.randint(0, E, (T, 1), device="cuda", generator=g).int()
    plan = [torch.empty(k, dtype=torch.int32, device="cuda") for k in (E, E + 1, T, T)]
    xq = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, d // 128, device="cuda")
    lib.moe_dispatch_fp8(x, idx, E, *plan, xq, xs, lib.workspace(lib.dispatch_ws_bytes(T, d, E, 1)))
    codes, scales = torch.empty_like(xq), torch.empty_like(xs)
    lib.moe_quantize_fp8(x[plan[2].long()], codes, scales)
    # zeros of a block of zeros keep their sign here
    empty = (scales == 0).repeat_interleave(128, 1)
    assert empty.any() and (codes[empty] & 0x7f == 0).all() and (xq[empty] == 0).all()
    assert torch.equal(codes[~empty], xq[~empty]) and torch.equal(scales, xs)
