"""GPU: edges of routing by scores, of the quantiser and of the products on block-scaled fp8."""
import numpy as np
import pytest
import torch

from tests import test_gpu_product_fp8 as products
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


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("pad", [0, 2])
def test_products_of_several_tiles_a_block(lib, back, pad):
    """Uneven segments of 116 row tiles and five column tiles (nine for the gradient): every
    resident block takes three tiles or more, of several experts."""
    g = np.random.default_rng(8)
    counts = [int(c) for c in g.integers(0, 640, 37)]
    counts[5] = counts[6] = counts[36] = 0
    counts[0] = 1
    for dtype in (torch.bfloat16, torch.float32, torch.float16):
        products.run_rows(lib, counts, 1040, 2064 if back else 656, dtype, back, tail=7, lead=2,
                          seed=3, pad=pad)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_router_of_more_tokens_than_a_pass_takes(lib, score):
    """Warps take a second and third token."""
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(45001, 64, device="cuda", generator=g)
    bias = torch.randn(64, device="cuda", generator=g) * 0.05
    for b in (None, bias):
        for kw in ({}, dict(groups=8, top_groups=3, group_keys=2)):
            routes.check(lib, x, b, 6, score=score, **kw)
    for renormalise in (True, False):
        routes.test_gradient(lib, 45001, 60, 3, score, renormalise, torch.float32)


def small_codes(shape, g):
    """Codes of every magnitude below 2, made without a copy in floats."""
    c = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    return c.bitwise_and_(0xbf).view(torch.float8_e4m3fn)


@pytest.mark.parametrize("back", [False, True])
def test_product_rows_past_32_bit_offsets(lib, back):
    """More than 2^31 elements in the matrix of codes, or in the result."""
    g = torch.Generator(device="cuda").manual_seed(9)
    N, n, K = (1 << 20) + 300, 16, 2064
    assert N * K > 1 << 31
    ends = [0, 1000, N - 700, N]
    inner, outer = (n, K) if back else (K, n)
    a, w = small_codes((N, inner), g), small_codes((3, n, K), g)
    sa = torch.rand(N, products.blocks(inner), device="cuda", generator=g) + 0.25
    sw = torch.rand(3, 1, products.blocks(K), device="cuda", generator=g) + 0.25
    out = torch.empty(N, outer, dtype=torch.bfloat16, device="cuda")
    f = lib.moe_product_fp8_dx if back else lib.moe_product_fp8
    f(a, sa, w, sw, out, lib.workspace(lib.product_fp8_ws_bytes(N, n, K, 3)),
      offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), flags=lib.MOE_CHECK)
    for e, at, end in ((0, 0, 1000), (1, 1000, 1500), (1, N // 2, N // 2 + 500),
                       (1, N - 1200, N - 700), (2, N - 700, N)):
        av = products.value(a[at:end], sa[at:end], "row")
        wv = products.value(w[e], sw[e], "tile")
        wv = wv if back else wv.t()
        products.within(out[at:end], av @ wv, av.abs() @ wv.abs(), inner, torch.bfloat16,
                        f"rows {at} to {end}")


@pytest.mark.parametrize("accumulate", [False, True])
def test_weights_gradients_past_32_bit_offsets(lib, accumulate):
    g = torch.Generator(device="cuda").manual_seed(10)
    E, n, K, N = 260, 2064, 4112, 256
    assert E * n * K > 1 << 31
    dy, x = small_codes((N, n), g), small_codes((N, K), g)
    sy, sx = (torch.rand(2, k, device="cuda", generator=g) + 0.25 for k in (n, K))
    ends = [0] + [128] * (E - 1) + [256]             # the first and the last expert have rows
    before = 0.5 if accumulate else float("nan")
    dw = torch.full((E, n, K), before, dtype=torch.bfloat16, device="cuda")
    lib.moe_product_fp8_dw(dy, sy, x, sx, dw, lib.workspace(lib.product_fp8_ws_bytes(N, n, K, E)),
                           offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"),
                           accumulate=accumulate, flags=lib.MOE_CHECK)
    assert (dw[1:-1] == (0.5 if accumulate else 0.0)).all()
    for e, b in ((0, 0), (E - 1, 1)):
        r = slice(128 * b, 128 * b + 128)
        yv = products.value(dy[r], sy[b:b + 1], "col").t()
        xv = products.value(x[r], sx[b:b + 1], "col")
        products.within(dw[e], yv @ xv, yv.abs() @ xv.abs(), 128, torch.bfloat16, f"expert {e}",
                        torch.full_like(yv @ xv, 0.5) if accumulate else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_between_other_columns(lib, dtype):
    """Logits and gradient as parts of wider matrices: what is beside them stays."""
    g = torch.Generator(device="cuda").manual_seed(13)
    for cut, E in ((slice(0, 64), 64), (slice(4, 68), 64), (slice(1, 61), 60)):
        wide = torch.randn(70, 80, device="cuda", generator=g).to(dtype)
        x = wide[:, cut]
        idx, _ = routes.forward(lib, x, None, 4, score="softmax")
        i64 = idx.cpu().numpy()
        dw = torch.randn(70, 4, device="cuda", generator=g)
        for score in ("sigmoid", "softmax"):
            for renormalise in (True, False):
                r = lib.Router(score=score, renormalise=renormalise)
                store = torch.full((70, 96), 3.0, device="cuda", dtype=dtype)
                lib.moe_route_scores_bwd(x, r, idx, dw, store[:, cut])
                a = [t.double().cpu().numpy() for t in (x, dw)]
                ref = routes.gradient(a[0], i64, a[1], score, renormalise, 1.0)
                size = routes.gradient_size(a[0], i64, a[1], score, renormalise, 1.0)
                # as test_gradient: expf, the sums over E and R, and the store
                slack = routes.UNIT * (np.ptp(a[0]) + E + 32) * size + 2.0 ** -50 * size.max()
                bound = slack + routes.HALF[dtype] * (np.abs(ref) + slack) + routes.TINY[dtype]
                assert (np.abs(store[:, cut].double().cpu().numpy() - ref) <= bound).all()
                store[:, cut] = 3.0
                assert (store == 3.0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_bias_of_nan_or_infinity_comes_first(lib, score):
    """The bias orders experts and takes no part in the weights."""
    x = torch.randn(40, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    want = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
    for bad in (float("nan"), float("inf")):
        bias = torch.zeros(64, device="cuda")
        bias[37] = bad
        for kw in ({}, dict(groups=4, top_groups=2), dict(groups=4, top_groups=1, group_keys=2)):
            idx, w = routes.forward(lib, x, bias, 6, score=score, renormalise=False, **kw)
            assert (idx[:, 0] == 37).all(), (bad, kw)
            got = want.gather(1, idx.long())
            # logits within 8 of each other, expf and a sum of 64: see test_gpu_route_scores
            assert ((w.double() - got).abs() <= routes.UNIT * (8 + 64 + 16) * got).all(), (bad, kw)


def test_split_products_follow_each_other_in_a_graph(lib):
    """Few tiles and a long contraction: parts of sums in the workspace and a second kernel.  One
    workspace for calls one after another, captured and replayed with other values."""
    g = torch.Generator(device="cuda").manual_seed(14)
    N, n, K = 3, 256, 4096
    x, sx = products.made((N, K), "row", g)
    w, sw = products.made((n, K), "tile", g)
    w2, sw2 = products.made((K, n), "tile", g)
    ws = lib.workspace(max(lib.product_fp8_ws_bytes(N, n, K), lib.product_fp8_ws_bytes(N, K, n)))
    assert ws.numel() > 256                       # split over several blocks
    a, b, c = (torch.empty(N, n, device="cuda") for _ in range(3))

    def step():
        lib.moe_product_fp8(x, sx, w, sw, a, ws)
        lib.moe_product_fp8_dx(x, sx, w2, sw2, b, ws)
        lib.moe_product_fp8(x, sx, w, sw, c, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        g.manual_seed(seed)
        x.copy_(products.made((N, K), "row", g)[0])
        sx.copy_(torch.rand(sx.shape, device="cuda", generator=g) + 0.25)
        for t in (a, b, c):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        xv, wv, w2v = (products.value(*p) for p in ((x, sx, "row"), (w, sw, "tile"),
                                                    (w2, sw2, "tile")))
        products.within(a, xv @ wv.t(), xv.abs() @ wv.abs().t(), K, torch.float32, "a")
        products.within(b, xv @ w2v, xv.abs() @ w2v.abs(), K, torch.float32, "b")
        assert torch.equal(a, c)
