"""GPU: expert sort (plan), rows to expert order and back, and their gradients,
against plain 64-bit computations.

Bounds.  One fp32 product rounds by 2^-24 of itself; the store rounds by half a
unit of the type (2^-8 bf16, 2^-11 fp16 with its subnormal step, 2^-24 fp32).  A
sum of k products in any order is within k * 2^-24 * sum |terms| of the exact one.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ULP = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
       torch.float32: (2.0 ** -24, 2.0 ** -150)}
EPS = 2.0 ** -24


def within(got, ref, bound, name):
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() > bound
    assert not over.any(), f"{name}: {int(over.sum())} off, worst {float((got - ref).abs().max())}"


def rounded(ref, terms, k, dtype):
    """Bound of a value that is a sum of k products with absolute terms `terms`, stored as dtype."""
    rel, tiny = ULP[dtype]
    slack = k * EPS * terms
    return slack + rel * (ref.abs() + slack) + tiny


def plan_reference(idx, E, align, capacity, N):
    """The plan, slot by slot."""
    flat = idx.reshape(-1)
    seen = np.zeros(E, np.int64)
    for e in flat:
        if 0 <= e < E:
            seen[e] += 1
    counts = np.minimum(seen, capacity) if capacity > 0 else seen
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    row_slot = np.full(N, -1, np.int64)
    slot_row = np.full(flat.size, -1, np.int64)
    at = np.zeros(E, np.int64)
    for s, e in enumerate(flat):
        if 0 <= e < E:
            if at[e] < counts[e]:
                row = offsets[e] + at[e]
                slot_row[s], row_slot[row] = row, s
            at[e] += 1
    return counts, offsets, row_slot, slot_row.reshape(idx.shape)


def sort(B, idx, E, align=1, capacity=0, extra=0, flags=None, stream=None):
    T, R = idx.shape
    N = B.sort_rows_bound(T, R, E, align, capacity) + extra
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.full((E,), -9, **i32), torch.full((E + 1,), -9, **i32), torch.full((N,), -9, **i32),
           torch.full((T, R), -9, **i32))
    B.moe_sort(idx, E, *out, B.workspace(B.sort_ws_bytes(T, E, R)), align=align,
               capacity=capacity, flags=B.MOE_CHECK if flags is None else flags, stream=stream)
    return out


def routing(T, E, R, seed, skew=0.0, empty=0.0):
    g = np.random.default_rng(seed)
    p = np.arange(1, E + 1, dtype=np.float64) ** -skew
    keys = np.log(p) - np.log(-np.log(g.random((T, E)).clip(1e-300, 1 - 1e-12)))
    idx = np.argsort(-keys, 1)[:, :R].astype(np.int32)
    idx[g.random((T, R)) < empty] = -1
    return idx


@pytest.mark.parametrize("T,E,R,align,capacity,empty,skew", [
    (0, 4, 2, 16, 0, 0.0, 0.0), (1, 1, 1, 1, 0, 0.0, 0.0), (1, 8, 2, 16, 0, 0.0, 0.0),
    (31, 5, 5, 3, 0, 0.2, 0.0), (33, 60, 3, 16, 0, 0.3, 0.0), (1000, 8, 2, 128, 100, 0.0, 1.0),
    (2731, 64, 3, 1, 0, 0.0, 1.2), (4096, 64, 6, 128, 300, 0.1, 1.0),
    (9000, 1024, 8, 16, 0, 0.05, 0.5), (40000, 256, 8, 1, 0, 0.0, 1.2)])
def test_plan(lib, T, E, R, align, capacity, empty, skew):
    idx = routing(T, E, R, seed=T + E, skew=skew, empty=empty)
    got = sort(lib, torch.from_numpy(idx).cuda(), E, align, capacity, extra=5)
    want = plan_reference(idx, E, align, capacity, got[2].numel())
    for name, g, w in zip(("counts", "offsets", "row_slot", "slot_row"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name


def test_plan_edges(lib):
    # no slot taken; one expert takes all; an expert twice in a token
    for idx in (np.full((700, 4), -1), np.full((700, 4), 2),
                np.random.default_rng(0).integers(0, 3, (5000, 7))):
        idx = idx.astype(np.int32)
        for align, cap in ((1, 0), (64, 0), (16, 33)):
            got = sort(lib, torch.from_numpy(idx).cuda(), 3, align, cap)
            want = plan_reference(idx, 3, align, cap, got[2].numel())
            for g, w in zip(got, want):
                assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("bad", [-2, 8, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("at", [0, 5000 * 4 - 1])
def test_bad_entries_are_reported_and_skipped(lib, bad, at):
    idx = routing(5000, 8, 4, seed=3)
    idx.reshape(-1)[at] = bad
    dev = torch.from_numpy(idx).cuda()
    with pytest.raises(lib.MoeError) as err:
        sort(lib, dev, 8)
    assert err.value.status == 4
    got = sort(lib, dev, 8, flags=0)
    want = plan_reference(idx, 8, 1, 0, got[2].numel())
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def spread_reference(x, w, slot_row, N):
    """rows and the absolute products, float64."""
    T, R = slot_row.shape
    rows = torch.zeros(N, x.shape[1], dtype=torch.float64, device=x.device)
    for r in range(R):
        t = (slot_row[:, r] >= 0).nonzero()[:, 0]
        rows[slot_row[t, r].long()] = x[t].double() * w[t, r, None].double()
    return rows


def collect_reference(rows, w, slot_row):
    """Sums, sums of absolute terms."""
    T, R = slot_row.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    a = torch.zeros_like(y)
    for r in range(R):
        t = (slot_row[:, r] >= 0).nonzero()[:, 0]
        term = rows[slot_row[t, r].long()].double() * w[t, r, None].double()
        y[t] += term
        a[t] += term.abs()
    return y, a


def dots_reference(tok, rows, slot_row):
    T, R = slot_row.shape
    dots = torch.zeros(T, R, dtype=torch.float64, device=rows.device)
    size = torch.zeros_like(dots)
    for r in range(R):
        t = (slot_row[:, r] >= 0).nonzero()[:, 0]
        term = tok[t].double() * rows[slot_row[t, r].long()].double()
        dots[t, r], size[t, r] = term.sum(1), term.abs().sum(1)
    return dots, size


def matrix(rows, d, dtype, gen, pad, shift, fill=None):
    """[rows, d] inside a wider buffer: row stride d + pad, first element at `shift`."""
    base = torch.randn(rows * (d + pad) + shift + 8, generator=gen, device="cuda").to(dtype)
    if fill is not None:
        base.fill_(fill)
    return base[shift:shift + rows * (d + pad)].view(rows, d + pad)[:, :d]


SHAPES = [  # T, d, E, R, align, capacity, empty, pad, shift
    (0, 64, 4, 2, 16, 0, 0.0, 0, 0), (1, 1, 1, 1, 1, 0, 0.0, 0, 0), (1, 7168, 8, 8, 16, 0, 0.0, 0, 0),
    (3, 8, 4, 2, 128, 0, 0.0, 0, 0), (37, 333, 6, 3, 1, 0, 0.3, 0, 0), (64, 130, 4, 2, 8, 20, 0.0, 2, 2),
    (100, 1024, 8, 2, 1, 0, 0.1, 24, 8), (129, 4096, 40, 32, 4, 0, 0.1, 0, 0),
    (300, 2050, 16, 11, 16, 0, 0.0, 1, 1), (2500, 512, 64, 6, 128, 200, 0.1, 0, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_and_gradients(lib, shape, dtype):
    T, d, E, R, align, capacity, empty, pad, shift = shape
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    idx = torch.from_numpy(routing(T, E, R, seed=T + d, skew=0.7, empty=empty)).cuda()
    _, _, row_slot, slot_row = sort(lib, idx, E, align, capacity, extra=3)
    N = row_slot.numel()
    x = matrix(T, d, dtype, gen, pad, shift)
    rows = matrix(N, d, dtype, gen, pad, shift)
    rows[row_slot < 0] = float("nan")                  # rows without a slot are never read
    w = torch.rand(T, R, generator=gen, device="cuda")
    w[slot_row < 0] = float("nan")                     # nor are the weights of empty slots
    one = torch.ones_like(w)
    live = row_slot >= 0
    for weight in (w, None):
        ww = w if weight is not None else one
        out = matrix(N, d, dtype, gen, pad, shift, fill=float("nan"))
        lib.moe_permute(x, weight, row_slot, slot_row, out)
        ref = spread_reference(x, ww, slot_row, N)
        within(out, ref, rounded(ref, ref.abs(), 1, dtype), "permute")
        assert (out[~live] == 0).all()
        if weight is None:
            assert torch.equal(out[live].float(), x[row_slot[live].long() // R].float())

        drows = matrix(N, d, dtype, gen, pad, shift, fill=float("nan"))
        dw = torch.full_like(w, float("nan"))
        lib.moe_unpermute_bwd(x, row_slot, slot_row, weight, rows, drows, dw)
        within(drows, ref, rounded(ref, ref.abs(), 1, dtype), "unpermute_bwd")
        assert (drows[~live] == 0).all()
        dots, size = dots_reference(x, rows, slot_row)
        within(dw, dots, (d + 1) * EPS * size + 1e-40, "dw")
        assert (dw[slot_row < 0] == 0).all()
        drows.fill_(float("nan"))
        lib.moe_unpermute_bwd(x, row_slot, slot_row, weight, None, drows, None)
        within(drows, ref, rounded(ref, ref.abs(), 1, dtype), "unpermute_bwd without dw")

        y = matrix(T, d, dtype, gen, pad, shift, fill=float("nan"))
        lib.moe_unpermute(rows, slot_row, weight, y)
        ref, terms = collect_reference(rows, ww, slot_row)
        within(y, ref, rounded(ref, terms, R + 1, dtype), "unpermute")
        assert (y[(slot_row < 0).all(1)] == 0).all()

        dx = matrix(T, d, dtype, gen, pad, shift, fill=float("nan"))
        dw.fill_(float("nan"))
        lib.moe_permute_bwd(rows, slot_row, weight, x, dx, dw)
        within(dx, ref, rounded(ref, terms, R + 1, dtype), "permute_bwd")
        within(dw, dots, (d + 1) * EPS * size + 1e-40, "dw")
        lib.moe_permute_bwd(rows, slot_row, weight, None, dx, None)
        within(dx, ref, rounded(ref, terms, R + 1, dtype), "permute_bwd without dw")


def test_neighbouring_memory_stays(lib):
    """The gaps between strided rows are not written."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    T, d, E, R = 50, 120, 4, 2
    idx = torch.from_numpy(routing(T, E, R, 1, empty=0.2)).cuda()
    _, _, row_slot, slot_row = sort(lib, idx, E, 16)
    wide = torch.full((row_slot.numel(), d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    lib.moe_permute(x, None, row_slot, slot_row, wide[:, :d])
    assert (wide[:, d:] == 7).all()
    y = torch.full((T, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.moe_unpermute(wide[:, :d], slot_row, None, y[:, :d])
    assert (y[:, d:] == 7).all()


def test_gradients_against_differences(lib):
    """Both directions are linear in rows and in weights, so central differences of a
    scalar loss are exact up to rounding: h = 1, fp32."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, d, E, R = 6, 40, 5, 3
    idx = torch.from_numpy(routing(T, E, R, 2, empty=0.2)).cuda()
    _, _, row_slot, slot_row = sort(lib, idx, E, 4)
    N = row_slot.numel()
    x = torch.randn(T, d, generator=gen, device="cuda")
    w = torch.rand(T, R, generator=gen, device="cuda")
    c_rows = torch.randn(N, d, generator=gen, device="cuda")
    c_y = torch.randn(T, d, generator=gen, device="cuda")
    rows_in = torch.randn(N, d, generator=gen, device="cuda")

    def loss_rows(x, w):
        rows = torch.empty(N, d, device="cuda")
        lib.moe_permute(x, w, row_slot, slot_row, rows)
        return float((rows.double() * c_rows.double()).sum())

    def loss_y(rows, w):
        y = torch.empty(T, d, device="cuda")
        lib.moe_unpermute(rows, slot_row, w, y)
        return float((y.double() * c_y.double()).sum())

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    lib.moe_permute_bwd(c_rows, slot_row, w, x, dx, dw)
    drows, dw2 = torch.empty_like(rows_in), torch.empty_like(w)
    lib.moe_unpermute_bwd(c_y, row_slot, slot_row, w, rows_in, drows, dw2)
    # |loss| sums N*d or T*d rounded terms: every one within 4 * 2^-24 of |values| <= ~20
    tol = 2 * 4 * EPS * 20 * N * d / 10
    for t in range(T):
        for r in range(R):
            e = torch.zeros_like(w)
            e[t, r] = 1.0
            assert abs((loss_rows(x, w + e) - loss_rows(x, w - e)) / 2 - float(dw[t, r])) < tol
            assert abs((loss_y(rows_in, w + e) - loss_y(rows_in, w - e)) / 2 - float(dw2[t, r])) < tol
    for k in range(0, T * d, 7):
        e = torch.zeros_like(x)
        e.view(-1)[k] = 1.0
        assert abs((loss_rows(x + e, w) - loss_rows(x - e, w)) / 2 - float(dx.view(-1)[k])) < tol
    for k in range(0, N * d, 13):
        e = torch.zeros_like(rows_in)
        e.view(-1)[k] = 1.0
        assert abs((loss_y(rows_in + e, w) - loss_y(rows_in - e, w)) / 2
                   - float(drows.view(-1)[k])) < tol


def test_same_bits_every_time_and_on_another_stream(lib):
    gen = torch.Generator(device="cuda").manual_seed(9)
    T, d, E, R = 3000, 776, 64, 6
    idx = torch.from_numpy(routing(T, E, R, 4, skew=1.0, empty=0.1)).cuda()
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    w = torch.rand(T, R, generator=gen, device="cuda")
    first = None
    for stream in (None, torch.cuda.Stream(), None):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            _, _, row_slot, slot_row = sort(lib, idx, E, 16)
            rows = torch.empty(row_slot.numel(), d, dtype=torch.bfloat16, device="cuda")
            dx, dw = torch.empty_like(x), torch.empty_like(w)
            lib.moe_permute(x, w, row_slot, slot_row, rows)
            lib.moe_permute_bwd(rows, slot_row, w, x, dx, dw)
        torch.cuda.synchronize()
        out = [row_slot, slot_row, rows.view(torch.int16), dx.view(torch.int16), dw]
        if first is None:
            first = out
        for a, b in zip(first, out):
            assert torch.equal(a, b)


def test_agrees_with_dispatch_and_combine(lib):
    """Without empty slots, limits or padding the plan is moe_dispatch's, the rows its
    copies and the sums moe_combine's, bit for bit."""
    T, d, E, R = 777, 256, 32, 4
    idx = torch.from_numpy(routing(T, E, R, 8)).cuda()
    counts, offsets, row_slot, slot_row = sort(lib, idx, E)
    x = torch.randn(T, d, device="cuda").bfloat16()
    w = torch.rand(T, R, device="cuda")
    rows = torch.empty(T * R, d, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    lib.moe_permute(x, None, row_slot, slot_row, rows)
    lib.moe_unpermute(rows, slot_row, w, y)
    other = [torch.empty_like(t) for t in (counts, offsets, row_slot, slot_row)]
    rows2, y2 = torch.empty_like(rows), torch.empty_like(y)
    lib.moe_dispatch(x, idx, E, *other, rows2, lib.workspace(lib.dispatch_ws_bytes(T, d, E, R)))
    lib.moe_combine(rows2, other[3], w, y2, R)
    for a, b in zip((counts, offsets, row_slot, slot_row, rows, y), (*other, rows2, y2)):
        assert torch.equal(a, b)


def test_capture(lib):
    """Plan, rows and gradients replay from a graph on new routing."""
    T, d, E, R = 200, 256, 16, 4
    idx = torch.from_numpy(routing(T, E, R, 1)).cuda()
    x = torch.randn(T, d, device="cuda").bfloat16()
    w = torch.rand(T, R, device="cuda")
    N = lib.sort_rows_bound(T, R, E, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(N, **i32),
            torch.empty((T, R), **i32))
    ws = lib.workspace(lib.sort_ws_bytes(T, E, R))
    rows, dx, dw = torch.empty(N, d, dtype=x.dtype, device="cuda"), torch.empty_like(x), torch.empty_like(w)

    def step():
        lib.moe_sort(idx, E, *plan, ws, align=16)
        lib.moe_permute(x, w, plan[2], plan[3], rows)
        lib.moe_permute_bwd(rows, plan[3], w, x, dx, dw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    idx.copy_(torch.from_numpy(routing(T, E, R, 2, empty=0.3)))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (*plan, rows, dx, dw)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, (*plan, rows, dx, dw)):
        assert torch.equal(a, b)


def test_rows_past_32_bit_offsets(lib):
    """More than 2^31 elements in the rows: the last tokens' copies, sums and gradients."""
    T, d, R = 40_000, 8192, 8
    idx = torch.arange(R, dtype=torch.int32, device="cuda").repeat(T, 1)
    _, _, row_slot, slot_row = sort(lib, idx, R)
    assert torch.equal(slot_row[-1], torch.arange(1, R + 1, device="cuda").int() * T - 1)
    x = torch.randn(T, d, device="cuda").bfloat16()
    rows = torch.empty(T * R, d, dtype=torch.bfloat16, device="cuda")
    lib.moe_permute(x, None, row_slot, slot_row, rows)
    for r in range(R):
        assert torch.equal(rows[r * T:(r + 1) * T], x)
    y, dw = torch.empty_like(x), torch.empty(T, R, device="cuda")
    lib.moe_permute_bwd(rows, slot_row, None, x, y, dw)
    assert torch.equal(y, (x.float() * R).bfloat16())           # sums of eight equal bf16 are exact
    exact = x[-100:].double().square().sum(1, keepdim=True)
    within(dw[-100:], exact.expand(-1, R), (d + 1) * EPS * exact, "dw")
