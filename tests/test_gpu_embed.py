"""GPU: embedding lookup and its gradient against 64-bit computations.

Bounds: the lookup is one fp32 product and one rounding; a gradient row of k
summands is within (k + 2) * 2^-24 * sum |terms| plus the rounding of the store.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_sort_rows import EPS, matrix, rounded, within

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def ids_of(n, V, kind, seed, dtype):
    g = np.random.default_rng(seed)
    if kind == "power":                                 # log-uniform: a few ids own most positions
        ids = np.exp(g.random(n) * np.log(V + 1)).astype(np.int64) - 1
        ids = np.clip(ids, 0, V - 1)
    elif kind == "one":
        ids = np.full(n, V - 1)
    elif kind == "none":
        ids = np.full(n, -1)
    elif kind == "distinct":
        ids = g.permutation(V)[:n]
    else:
        ids = g.integers(0, V, n)
    if kind == "masked":
        ids[g.random(n) < 0.3] = -7
    return torch.from_numpy(ids.astype(np.int64)).to(dtype).cuda()


CASES = [  # n, V, d, ids, pad, shift
    (1, 1, 1, "uniform", 0, 0), (1, 50000, 64, "uniform", 0, 0), (5, 3, 9, "masked", 0, 0),
    (64, 7, 256, "one", 0, 0), (65, 7, 1000, "one", 8, 8), (300, 513, 130, "masked", 2, 2),
    (1000, 40, 2048, "power", 0, 0), (777, 777, 72, "distinct", 0, 0), (100, 64, 24, "none", 0, 0),
    (4097, 70001, 40, "power", 0, 0), (20000, 300, 88, "power", 0, 0), (6000, 1500, 4100, "power", 0, 0)]


@pytest.mark.parametrize("types", [(BF, BF), (BF, F), (HF, HF), (F, F), (F, BF), (HF, F)])
@pytest.mark.parametrize("case", CASES)
def test_lookup_and_gradient(lib, case, types):
    n, V, d, kind, pad, shift = case
    source, dest = types
    gen = torch.Generator(device="cuda").manual_seed(n + V)
    ids = ids_of(n, V, kind, n + d, torch.int64 if n % 2 else torch.int32)
    long_ids = ids.long()
    live = (long_ids >= 0) & (long_ids < V)
    scale = 0.37
    table = matrix(V, d, source, gen, pad, shift)
    out = matrix(n, d, dest, gen, pad, shift, fill=float("nan"))
    lib.moe_embed(ids, table, out, scale=scale)
    f32 = float(np.float32(scale))
    ref = torch.where(live[:, None], table.double()[long_ids.clamp(0, V - 1)] * f32, 0.0)
    within(out, ref, rounded(ref, ref.abs(), 1, dest), "lookup")
    assert (out[~live] == 0).all()

    dout = matrix(n, d, source, gen, pad, shift)
    dout[~live] = float("nan")                          # positions without a token are not read
    sums = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(sums)
    sums.index_add_(0, long_ids[live], dout[live].double())
    size.index_add_(0, long_ids[live], dout[live].double().abs())
    count = torch.bincount(long_ids[live], minlength=V)[:, None].double()
    ws = lib.workspace(lib.embed_bwd_ws_bytes(n, V, d))
    grad = matrix(V, d, dest, gen, pad, shift, fill=float("nan"))
    lib.moe_embed_bwd(dout, ids, grad, ws, scale=scale, flags=lib.MOE_CHECK)
    ref, terms = sums * f32, size * f32
    within(grad, ref, rounded(ref, terms, count + 2, dest), "gradient")
    assert (grad[count[:, 0] == 0] == 0).all()

    grad = matrix(V, d, dest, gen, pad, shift)
    before = grad.clone()
    lib.moe_embed_bwd(dout, ids, grad, ws, scale=scale, accumulate=True, flags=lib.MOE_CHECK)
    ref, terms = before.double() + ref, before.double().abs() + terms
    within(grad, ref, rounded(ref, terms, count + 3, dest), "accumulated")
    untouched = count[:, 0] == 0
    assert torch.equal(grad[untouched], before[untouched])


def test_ids_past_the_table(lib):
    V, d, n = 100, 64, 500
    ids = torch.arange(n, device="cuda") % V
    dout = torch.randn(n, d, device="cuda")
    good = torch.empty(V, d, device="cuda")
    ws = lib.workspace(lib.embed_bwd_ws_bytes(n, V, d))
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[3, 77]] = False
    lib.moe_embed_bwd(dout[keep], ids[keep], good, ws, flags=lib.MOE_CHECK)
    for bad in (V, 2 ** 40, 2 ** 62):
        some = ids.clone()
        some[3], some[77] = bad, -2 ** 50
        got = torch.full((V, d), float("nan"), device="cuda")
        with pytest.raises(lib.MoeError) as err:
            lib.moe_embed_bwd(dout, some, got, ws, flags=lib.MOE_CHECK)
        assert err.value.status == 4
        assert torch.equal(got, good)
        out = torch.empty(n, d, device="cuda")
        lib.moe_embed(some, good, out)
        assert (out[3] == 0).all() and (out[77] == 0).all() and torch.equal(out[4], good[4])
    lib.moe_embed_bwd(dout, ids, got, ws, flags=lib.MOE_CHECK)     # the error word starts clean


def test_no_positions(lib):
    V, d = 10, 64
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    dout = torch.empty(0, d, device="cuda")
    grad = torch.full((V, d), 3.0, device="cuda")
    ws = lib.workspace(lib.embed_bwd_ws_bytes(0, V, d))
    lib.moe_embed_bwd(dout, ids, grad, ws, accumulate=True, flags=lib.MOE_CHECK)
    assert (grad == 3).all()
    lib.moe_embed_bwd(dout, ids, grad, ws, flags=lib.MOE_CHECK)
    assert (grad == 0).all()
    lib.moe_embed(ids, grad, dout)


def test_gradient_against_differences(lib):
    """The lookup is linear in the table: central differences with h = 1 are exact up to rounding."""
    n, V, d, scale = 90, 12, 24, 1.5
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = ids_of(n, V, "masked", 2, torch.int64)
    table = torch.randn(V, d, generator=gen, device="cuda")
    c = torch.randn(n, d, generator=gen, device="cuda")

    def loss(table):
        out = torch.empty(n, d, device="cuda")
        lib.moe_embed(ids, table, out, scale=scale)
        return float((out.double() * c.double()).sum())

    grad = torch.empty_like(table)
    lib.moe_embed_bwd(c, ids, grad, lib.workspace(lib.embed_bwd_ws_bytes(n, V, d)), scale=scale)
    for k in range(0, V * d, 5):
        e = torch.zeros_like(table)
        e.view(-1)[k] = 1.0
        # n terms of |scale * table * c| <= 30, each rounded by 2^-24 on either side
        assert abs((loss(table + e) - loss(table - e)) / 2 - float(grad.view(-1)[k])) < 4 * n * 30 * EPS


def test_same_bits_every_time(lib):
    n, V, d = 30000, 5000, 264
    ids = ids_of(n, V, "power", 3, torch.int32)
    dout = torch.randn(n, d, device="cuda").bfloat16()
    first = None
    for _ in range(3):
        ws = torch.randint(0, 255, (lib.embed_bwd_ws_bytes(n, V, d),), dtype=torch.uint8, device="cuda")
        grad = torch.empty(V, d, device="cuda")
        lib.moe_embed_bwd(dout, ids, grad, ws)
        first = grad if first is None else first
        assert torch.equal(first, grad)


@pytest.mark.parametrize("accumulate", [False, True])
def test_capture(lib, accumulate):
    """Lookup and gradient replay from a graph on new ids."""
    n, V, d = 3000, 700, 320
    ids = ids_of(n, V, "power", 1, torch.int64)
    table = torch.randn(V, d, device="cuda").bfloat16()
    dout = torch.randn(n, d, device="cuda").bfloat16()
    out, grad = torch.empty(n, d, dtype=BF, device="cuda"), torch.zeros(V, d, device="cuda")
    ws = lib.workspace(lib.embed_bwd_ws_bytes(n, V, d))

    def step():
        lib.moe_embed(ids, table, out, scale=2.0)
        lib.moe_embed_bwd(dout, ids, grad, ws, accumulate=accumulate)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ids.copy_(ids_of(n, V, "masked", 2, torch.int64))
    grad.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = [out.clone(), grad.clone()]
    grad.zero_()
    step(), step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], grad)


def test_table_past_32_bit_offsets(lib):
    """More than 2^31 elements in the table: lookup and gradient at its end."""
    V, d = 600_001, 4096
    table = torch.empty(V, d, dtype=BF, device="cuda")
    table[-3:] = torch.randn(3, d, device="cuda").bfloat16()
    ids = torch.tensor([V - 1, V - 3, V - 1, V - 2], device="cuda")
    out = torch.empty(4, d, dtype=BF, device="cuda")
    lib.moe_embed(ids, table, out)
    assert torch.equal(out, table[ids])
    grad = torch.full((V, d), float("nan"), dtype=BF, device="cuda")
    lib.moe_embed_bwd(out, ids, grad, lib.workspace(lib.embed_bwd_ws_bytes(4, V, d)),
                      flags=lib.MOE_CHECK)
    assert torch.equal(grad[-2:], torch.stack([out[3], (out[0].float() * 2).bfloat16()]))
    assert torch.equal(grad[-3], out[1])
    for rows in grad[:-3].split(100_000):
        assert not rows.any()
