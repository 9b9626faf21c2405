"""GPU: routing by scores and its gradient against plain 64-bit computations.

Bounds.  expf is within 2 units (2^-23 each) of the exponential of its argument; an argument
y - top rounds by 2^-24 of itself, which the exponential turns into a relative error; a sum of k
terms adds k units of 2^-24, products and quotients one each.  With logits within D of each other a
weight is within 2^-23 (D + k + 16) of itself.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
UNIT = 2.0 ** -23


def scores(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(1, keepdims=True)
    z = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    return z / np.maximum(z.sum(1, keepdims=True), 1e-300)


def choice(x, bias, R, score, groups=1, top_groups=1, group_keys=1):
    """The definition, in 64 bits."""
    T, E = x.shape
    s = scores(x, score)
    key = s + bias if bias is not None else s
    by = key if bias is not None else x
    worth_key = key if bias is not None or group_keys == 2 else x
    closed = x == -np.inf
    by, worth_key = (np.where(closed, -np.inf, v) for v in (by, worth_key))
    if groups > 1:
        per = E // groups
        best = -np.sort(-worth_key.reshape(T, groups, per), axis=2)[:, :, :group_keys]
        place = np.argsort(-best.sum(2), axis=1, kind="stable")[:, :top_groups]
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, place, True, 1)
        by = np.where(np.repeat(keep, per, 1), by, -np.inf)
    idx = np.argsort(-by, axis=1, kind="stable")[:, :R]
    return np.where(np.take_along_axis(by, idx, 1) == -np.inf, -1, idx)


def weights(x, idx, score, renormalise, scale):
    s = np.take_along_axis(scores(x, score), np.maximum(idx, 0), 1)
    s = np.where(idx >= 0, s, 0.0)
    if renormalise:
        s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
    return s * scale


def gradient(x, idx, dw, score, renormalise, scale):
    T, E = x.shape
    s = scores(x, score)
    here = (idx >= 0) & (idx < E)
    at = np.where(here, idx, 0)
    here &= np.take_along_axis(x, at, 1) > -np.inf
    g = np.where(here, dw, 0.0) * scale
    chosen = np.where(here, np.take_along_axis(s, at, 1), 0.0)
    if renormalise:
        total = np.maximum(chosen.sum(1, keepdims=True), 1e-300)
        u = chosen / total
        g = np.where(here, (g - (g * u).sum(1, keepdims=True)) / total, 0.0)
    ds = np.zeros((T, E))
    np.add.at(ds, (np.arange(T)[:, None], at), g)
    if score == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(1, keepdims=True))


def forward(lib, x, bias, R, **router):
    T = x.shape[0]
    idx = torch.full((T, R), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, R), float("nan"), device="cuda")
    lib.moe_route_scores(x, lib.Router(**router), idx, w, bias=bias)
    return idx, w


def check(lib, x, bias, R, score="sigmoid", groups=1, top_groups=1, group_keys=1, renormalise=True,
          scale=1.0):
    idx, w = forward(lib, x, bias, R, score=score, groups=groups, top_groups=top_groups,
                     group_keys=group_keys, renormalise=renormalise, scale=scale)
    x64 = x.double().cpu().numpy()
    b64 = None if bias is None else bias.double().cpu().numpy()
    ref = choice(x64, b64, R, score, groups, top_groups, group_keys)
    got = idx.cpu().numpy()
    assert np.array_equal(got, ref), f"{(got != ref).any(1).sum()} tokens of {len(ref)}"
    want = weights(x64, ref, score, renormalise, scale)
    finite = x64[np.isfinite(x64)]
    D = finite.max() - finite.min() if finite.size else 0.0
    bound = UNIT * (D + x.shape[1] + 16) * want + 2.0 ** -140
    off = np.abs(w.double().cpu().numpy() - want)
    assert (off <= bound).all(), f"weights off by {(off / np.maximum(bound, 1e-300)).max()} bounds"
    return idx, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,R", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (257, 8, 2), (100, 33, 5),
                                   (64, 60, 3), (1000, 128, 8), (513, 160, 6), (300, 256, 8),
                                   (200, 384, 8), (77, 512, 32), (40, 1000, 7), (33, 1024, 32)])
def test_plain_routing(lib, T, E, R, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn(T, E, device="cuda", generator=g).to(dtype)
    bias = torch.randn(E, device="cuda", generator=g) * 0.05
    for score in ("sigmoid", "softmax"):
        for b in (None, bias):
            check(lib, x, b, R, score=score, renormalise=b is None, scale=2.5)
            check(lib, x, b, R, score=score, renormalise=b is not None)


@pytest.mark.parametrize("T,E,R,groups,top_groups", [
    (128, 256, 8, 8, 4), (500, 256, 8, 8, 1), (9, 64, 4, 32, 3), (300, 160, 6, 8, 3),
    (200, 60, 3, 5, 2), (150, 200, 8, 4, 2), (111, 66, 5, 3, 1), (70, 1024, 8, 16, 16),
    (64, 96, 20, 3, 2), (50, 62, 4, 31, 30)])
def test_groups(lib, T, E, R, groups, top_groups):
    g = torch.Generator(device="cuda").manual_seed(E)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(T, E, device="cuda", generator=g).to(dtype)
        bias = torch.randn(E, device="cuda", generator=g) * 0.05
        for score in ("sigmoid", "softmax"):
            for keys in (1, 2):
                for b in (None, bias):
                    check(lib, x, b, R, score=score, groups=groups, top_groups=top_groups,
                          group_keys=keys)


def test_keys_closer_than_32_bits(lib):
    """Pairs whose keys differ by less than 2^-25: the order is that of 64 bits."""
    g = np.random.default_rng(5)
    E = 64
    x = g.normal(size=(4096, E)).astype(np.float32)
    bias = (g.normal(size=E) * 0.05).astype(np.float32)
    # the second half of each token's experts almost ties with the first half
    want = scores(x[:, :32].astype(np.float64), "sigmoid") + bias[:32] - bias[32:]
    want = want.clip(1e-3, 1 - 1e-3)
    x[:, 32:] = np.log(want / (1 - want)).astype(np.float32)
    perm = g.permutation(E)
    x, bias = np.ascontiguousarray(x[:, perm]), np.ascontiguousarray(bias[perm])
    xd, bd = torch.from_numpy(x).cuda(), torch.from_numpy(bias).cuda()
    for R in (1, 7, 8):
        check(lib, xd, bd, R)
        check(lib, xd, bd, R, groups=8, top_groups=4, group_keys=2)
        check(lib, xd, bd, R, groups=8, top_groups=3, group_keys=1)


def test_ties_go_to_the_lower_expert_and_group(lib):
    x = torch.zeros(5, 96, device="cuda")
    x[1:, 40:] = 1.0
    x[2, ::3] = -0.0
    bias = torch.zeros(96, device="cuda")
    for b in (None, bias):
        for score in ("sigmoid", "softmax"):
            check(lib, x, b, 8, score=score)
            check(lib, x, b, 8, score=score, groups=6, top_groups=2, group_keys=2)
    idx, _ = forward(lib, x, None, 8, score="softmax")
    assert idx[0].tolist() == list(range(8)) and idx[1].tolist() == list(range(40, 48))


def test_closed_experts(lib):
    inf = float("inf")
    x = torch.randn(64, 48, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[:16] = -inf                       # nothing open
    x[16:32, 3:] = -inf                 # fewer open than slots
    x[32:, ::2] = -inf
    for score in ("sigmoid", "softmax"):
        for renormalise in (True, False):
            for groups in (1, 4):
                idx, w = check(lib, x, None, 6, score=score, renormalise=renormalise,
                               groups=groups, top_groups=max(1, groups // 2),
                               group_keys=2 if groups > 1 else 1)
                assert (idx[:16] == -1).all() and (w[:16] == 0).all()
    bias = torch.zeros(48, device="cuda")
    bias[1] = -inf
    idx, _ = forward(lib, x, bias, 6, score="sigmoid")
    assert not (idx == 1).any()


def test_wide_logits(lib):
    """Scores far below the fp32 range still share their weight."""
    x = torch.tensor([[-300.0, -299.0, -310.0, -1000.0], [90.0, 89.0, -500.0, 30.0]], device="cuda")
    for score in ("sigmoid", "softmax"):
        idx, w = forward(lib, x, None, 2, score=score, renormalise=True)
        assert idx.tolist() == [[1, 0], [0, 1]]
    _, w = forward(lib, x, None, 2, score="sigmoid", renormalise=True)
    share = 1.0 / (1.0 + np.exp(-1.0))
    assert abs(float(w[0, 0]) - share) < 64 * UNIT and abs(float(w[1, 0]) - 0.5) < 64 * UNIT


def test_nan_is_seen(lib):
    x = torch.zeros(4, 64, device="cuda")
    x[1, 37] = float("nan")
    x[2] = float("nan")
    x[3, 5] = float("inf")
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.zeros(64, device="cuda")):
            for groups in (1, 4):
                idx, w = forward(lib, x, bias, 3, score=score, groups=groups,
                                 top_groups=max(1, groups // 2))
                assert torch.isfinite(w[0]).all() and torch.isnan(w[2]).all()
                assert idx[2].tolist() == [0, 1, 2]
                if score == "sigmoid" or bias is None:
                    assert int(idx[1, 0]) == 37 and torch.isnan(w[1, 0])
                    assert int(idx[3, 0]) == 5
                else:       # a softmax over a NaN is NaN throughout
                    assert torch.isnan(w[1]).any() or int(idx[1, 0]) == 0


def test_strided_rows_and_streams(lib):
    g = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.randn(50, 300, device="cuda", generator=g)
    for cut in (slice(0, 256), slice(1, 257), slice(3, 131)):
        check(lib, wide[:, cut], None, 8, score="softmax", renormalise=False)
    x = wide[:, :128].contiguous()
    s = torch.cuda.Stream()
    idx = torch.empty(50, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(50, 4, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    lib.moe_route_scores(x, lib.Router(score="sigmoid"), idx, w, stream=s)
    s.synchronize()
    again = forward(lib, x, None, 4, score="sigmoid")
    assert torch.equal(idx, again[0]) and torch.equal(w, again[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,R", [(1, 1, 1), (2, 256, 8), (300, 128, 8), (65, 60, 3),
                                   (129, 384, 6), (31, 1000, 32)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient(lib, T, E, R, score, renormalise, dtype):
    g = torch.Generator(device="cuda").manual_seed(T * E)
    x = (torch.randn(T, E, device="cuda", generator=g) * 2).to(dtype)
    if E > R + 2:
        x[:, 1] = -float("inf")
    scale = 2.5
    idx, _ = forward(lib, x, None, R, score=score)
    idx[T // 2, R // 2] = -1
    dw = torch.randn(T, R, device="cuda", generator=g)
    dw[T // 2, R // 2] = float("nan")              # not read
    out = torch.full((T, E), float("nan"), device="cuda", dtype=dtype)
    lib.moe_route_scores_bwd(x, lib.Router(score=score, renormalise=renormalise, scale=scale), idx,
                             dw, out)
    x64, i64, d64 = x.double().cpu().numpy(), idx.cpu().numpy(), dw.double().cpu().numpy()
    ref = gradient(x64, i64, d64, score, renormalise, scale)
    # terms: what cancels in g - sum g u, at the size of the parts
    big = gradient_size(x64, i64, d64, score, renormalise, scale)
    D = np.ptp(x64[np.isfinite(x64)])
    slack = UNIT * (D + E + 32) * big
    bound = slack + HALF[dtype] * (np.abs(ref) + slack) + TINY[dtype]
    # the reference's own rounding: a softmax's ds - sum ds s cancels to exactly 0 for experts that
    # renormalised weights do not depend on, in 64 bits to R + 4 units of 2^-53 of the sum's parts
    if score == "softmax":
        s64 = scores(x64, score)
        ds = big / np.maximum(s64, 1e-300)
        bound += (R + 4) * 2.0 ** -52 * s64 * (ds * s64).sum(1, keepdims=True)
    off = np.abs(out.double().cpu().numpy() - ref)
    assert np.isfinite(out.float().cpu().numpy()).all()
    assert (off <= bound).all(), f"off by {(off / bound).max()} bounds"


def gradient_size(x, idx, dw, score, renormalise, scale):
    """The gradient with every term's magnitude."""
    T, E = x.shape
    s = scores(x, score)
    here = idx >= 0
    at = np.maximum(idx, 0)
    here = here & (np.take_along_axis(x, at, 1) > -np.inf)
    g = np.abs(np.where(here, np.nan_to_num(dw), 0.0) * scale)
    chosen = np.where(here, np.take_along_axis(s, at, 1), 0.0)
    if renormalise:
        total = np.maximum(chosen.sum(1, keepdims=True), 1e-300)
        g = np.where(here, (g + (g * chosen / total).sum(1, keepdims=True)) / total, 0.0)
    ds = np.zeros((T, E))
    np.add.at(ds, (np.arange(T)[:, None], at), g)
    if score == "sigmoid":
        return ds * s * (1.0 - s)
    if renormalise:
        return s * ds
    return s * (ds + (ds * s).sum(1, keepdims=True))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient_against_differences(lib, score, renormalise):
    """The formula of the test itself, against central differences of the weights (64 bits):
    the third derivative of a score is below 1, so a step of 1e-4 leaves below 1e-7."""
    g = np.random.default_rng(2)
    x = g.normal(size=(4, 12))
    idx = np.argsort(-x, 1)[:, :3]
    dw = g.normal(size=(4, 3))
    ref = gradient(x, idx, dw, score, renormalise, 2.5)
    h = 1e-4
    for e in range(12):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        diff = (weights(up, idx, score, renormalise, 2.5)
                - weights(down, idx, score, renormalise, 2.5)) / (2 * h)
        assert np.abs((diff * dw).sum(1) - ref[:, e]).max() < 1e-6


def test_gradient_of_an_expert_named_twice(lib):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(40, 64, device="cuda", generator=g)
    idx = torch.randint(0, 3, (40, 5), device="cuda", generator=g).int()
    idx[0] = torch.tensor([7, 64, -1, 7, 1000])          # outside: contributes nothing
    dw = torch.randn(40, 5, device="cuda", generator=g)
    for score in ("sigmoid", "softmax"):
        for renormalise in (True, False):
            out = torch.empty(40, 64, device="cuda")
            lib.moe_route_scores_bwd(x, lib.Router(score=score, renormalise=renormalise), idx, dw,
                                     out)
            ref = gradient(x.double().cpu().numpy(), idx.cpu().numpy(),
                           dw.double().cpu().numpy(), score, renormalise, 1.0)
            assert np.abs(out.double().cpu().numpy() - ref).max() < UNIT * 128 * 16


def test_replayed_graph_follows_its_inputs(lib):
    x = torch.randn(64, 256, device="cuda")
    bias = torch.zeros(256, device="cuda")
    dw = torch.randn(64, 8, device="cuda")
    idx = torch.empty(64, 8, dtype=torch.int32, device="cuda")
    w, dl = torch.empty(64, 8, device="cuda"), torch.empty_like(x)
    r = lib.Router(score="sigmoid", groups=8, top_groups=4, group_keys=2)

    def step():
        lib.moe_route_scores(x, r, idx, w, bias=bias)
        lib.moe_route_scores_bwd(x, r, idx, dw, dl)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn(64, 256, device="cuda"))
    bias.copy_(torch.randn(256, device="cuda") * 0.1)
    graph.replay()
    torch.cuda.synchronize()
    got = idx.clone(), w.clone(), dl.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], idx) and torch.equal(got[1], w) and torch.equal(got[2], dl)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient_of_closed_tokens_is_zero(lib, score, renormalise):
    """Every expert closed (a padded token), or the chosen ones alone."""
    x = torch.randn(6, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[:2] = -float("inf")
    x[2, :4] = -float("inf")
    idx = torch.arange(4, device="cuda").int().repeat(6, 1)
    idx[0] = -1
    dw = torch.ones(6, 4, device="cuda")
    out = torch.full((6, 64), float("nan"), device="cuda")
    lib.moe_route_scores_bwd(x, lib.Router(score=score, renormalise=renormalise), idx, dw, out)
    assert torch.isfinite(out).all()
    assert (out[:3] == 0).all()
    if renormalise:     # equal dw: the weights' sum is fixed, so the gradient is 0 but for rounding
        assert (out[3:].abs() <= 64 * 2.0 ** -24).all()
    else:
        assert (out[3:] != 0).any(1).all()


def test_logits_and_biases_of_any_range(lib):
    """Keys whose range leaves the steps of a key's integer, or fp32 altogether."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(40, 96, device="cuda", generator=g)
    x[::4] *= 1e-6
    x[1::4] *= 1e30
    x[2::4, ::2] = 3e38
    x[2::4, 1::2] = -3e38
    for score in ("sigmoid", "softmax"):
        idx, _ = forward(lib, x, None, 8, score=score)
        assert np.array_equal(idx.cpu().numpy(), choice(x.double().cpu().numpy(), None, 8, score))
    x = torch.randn(40, 96, device="cuda", generator=g)
    for size in (1e-8, 1e3, 1e20, 1e35):
        bias = torch.randn(96, device="cuda", generator=g) * size
        idx, _ = forward(lib, x, bias, 8, score="sigmoid")
        ref = choice(x.double().cpu().numpy(), bias.double().cpu().numpy(), 8, "sigmoid")
        assert np.array_equal(idx.cpu().numpy(), ref), size


def test_a_long_run_of_near_ties(lib):
    """More keys within the error bound of each other than a warp has lanes: all of the token's
    choice in 64 bits.  Logits of 20 to 30 have sigmoids within 2e-9 of each other."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.rand(20, 256, device="cuda", generator=g) * 10 + 20
    x[::2, 100:] -= 30
    bias = torch.zeros(256, device="cuda")
    for groups in (1, 8):
        check(lib, x, bias, 8, groups=groups, top_groups=max(1, groups // 2),
              group_keys=2 if groups > 1 else 1)


@pytest.mark.parametrize("E,R", [(96, 8), (384, 8), (64, 1), (1024, 32), (256, 20)])
def test_equal_keys_beside_closer_ones(lib, E, R):
    """Few values and their neighbours in fp32, many times over, beside one far below: equal keys
    lie between others that the token's range does not tell apart."""
    g = np.random.default_rng(E + R)
    values = np.array([2.5, 2.25, 1.75, 0.5], np.float32)
    x = values[g.integers(0, g.integers(1, 5, (512, 1)), (512, E))]
    step = g.integers(-2, 3, (512, E)) * (g.random((512, 1)) < 0.7)
    x = (x.view(np.int32) + step.astype(np.int32)).view(np.float32)
    x[:, 0] = -9.0
    x = torch.from_numpy(x).cuda()
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.full((E,), 0.25, device="cuda")):
            check(lib, x, bias, R, score=score)


@pytest.mark.parametrize("E,groups,top_groups", [(256, 8, 4), (1024, 4, 1), (62, 31, 20), (96, 6, 5),
                                                 (64, 32, 9)])
def test_groups_closer_than_32_bits(lib, E, groups, top_groups):
    """Groups that are others' copies, some a unit of 2^-24 off or exact: their worths differ by
    less than 32 bits tell, or tie; in some tokens fewer groups are open than may take part."""
    g = np.random.default_rng(E)
    T, per = 512, E // groups
    x = g.normal(size=(T, groups, per)).astype(np.float32)
    for t in range(T):
        of = g.integers(0, groups, groups) if t % 3 else np.zeros(groups, int)
        x[t] = x[t, of]
        step = g.integers(-1, 2, (groups, 1))
        x[t] = np.where(step == 0, x[t], np.nextafter(x[t], np.float32(9) * step.astype(np.float32)))
        if t % 5 == 0:
            x[t, g.permutation(groups)[:groups // 2]] = -np.inf
        if t % 7 == 0:
            x[t, :, g.integers(0, per)] = -np.inf
    x = torch.from_numpy(np.ascontiguousarray(x.reshape(T, E))).cuda()
    R = min(8, per * top_groups)
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.full((E,), 0.25, device="cuda")):
            for keys in (1, 2):
                check(lib, x, bias, R, score=score, groups=groups, top_groups=top_groups,
                      group_keys=keys)


@pytest.mark.parametrize("size", [-3e7, 1e4, 3e7, 1e9, 1e29, 3e38])
def test_large_biases_that_hardly_differ(lib, size):
    """A bias that is far above the scores, for all experts or all but a step of fp32: what is
    left of the scores in 64 bits decides."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(200, 128, device="cuda", generator=g)
    bias = torch.full((128,), size, device="cuda")
    for groups in (1, 4):
        kw = dict(groups=groups, top_groups=max(1, groups // 2), group_keys=2 if groups > 1 else 1)
        check(lib, x, bias, 8, **kw)
        some = bias.view(torch.int32) - torch.arange(128, device="cuda", dtype=torch.int32) % 3
        check(lib, x, some.view(torch.float32), 8, **kw)
