"""GPU: the experts' products on block-scaled fp8 against 64-bit products of the decoded values.

Bounds.  Products of two codes are exact in fp32.  The tensor cores add the 32 products of a step
and the accumulator with at least 24 bits below the largest of them: an error of at most
33 * 2^-23 of the terms' magnitudes a step, four steps a block.  A block's scale (a product of two)
and its fma round by 2^-24 each, as does each addition of a split's part.  With A the sum of the
terms' magnitudes the fp32 result is within (132 + 3 blocks + 160) * 2^-23 A, and the store rounds
by half a unit of the type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // 128)


def made(shape, form, g, scale=1.0):
    """Random codes over the whole range of magnitudes, random scales."""
    codes = torch.randn(shape, device="cuda", generator=g).mul_(60).clamp_(-448, 448).to(E4M3)
    n, K = shape[-2:]
    s = shape[:-2] + ((n if form == "row" else blocks(n)), (K if form == "col" else blocks(K)))
    return codes, torch.rand(s, device="cuda", generator=g).add_(0.25).mul_(scale)


def value(codes, scales, form):
    n, K = codes.shape[-2:]
    v = scales.double()
    if form != "row":
        v = v.repeat_interleave(128, -2)[..., :n, :]
    if form != "col":
        v = v.repeat_interleave(128, -1)[..., :K]
    return codes.double() * v


def within(got, ref, size, k, dtype, name, extra=None):
    slack = (292 + 3 * blocks(k)) * 2.0 ** -23 * size
    if extra is not None:
        slack = slack + 2.0 ** -24 * (size + extra.abs())
        ref = ref + extra
    bound = slack + HALF[dtype] * (ref.abs() + slack) + TINY[dtype]
    got = got.double()
    assert torch.isfinite(got).all(), name
    off = (got - ref).abs() / bound
    assert float(off.max()) <= 1.0, f"{name}: off by {float(off.max())} bounds"


def segments(counts, align=1):
    offsets, at = [0], 0
    for c in counts:
        at += -(-c // align) * align
        offsets.append(at)
    return offsets


def run_rows(lib, counts, n, K, dtype, back, tail=0, lead=0, seed=0, pad=0, flags=None):
    """PRODUCT or PRODUCT_DX over segments; everything outside the segments is NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    ends = [lead + o for o in segments(counts)]
    N = ends[-1] + tail
    inner, outer = (n, K) if back else (K, n)
    a, sa = made((N, inner), "row", g)
    w, sw = made((E, n, K), "tile", g, 1e-3)
    a.view(torch.uint8)[:lead] = 0x7f
    a.view(torch.uint8)[ends[-1]:] = 0x7f
    sa[:lead] = float("nan")
    sa[ends[-1]:] = float("nan")
    for e, c in enumerate(counts):
        if c == 0:                                   # weights that no row uses
            w[e].view(torch.uint8).fill_(0x7f)
            sw[e] = float("nan")
    store = torch.full((N, outer + pad), -7.0, device="cuda", dtype=dtype)
    out = store[:, pad // 2:pad // 2 + outer]
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    f = lib.moe_product_fp8_dx if back else lib.moe_product_fp8
    ws = lib.workspace(lib.product_fp8_ws_bytes(N, n, K, E))
    ws.fill_(0xff)
    f(a, sa, w, sw, out, ws, offsets=offsets, flags=lib.MOE_CHECK if flags is None else flags)
    assert (out[:lead] == -7.0).all() and (out[ends[-1]:] == -7.0).all()
    if pad:
        assert (store[:, :pad // 2] == -7.0).all() and (store[:, pad // 2 + outer:] == -7.0).all()
    for e in range(E):
        i = slice(ends[e], ends[e + 1])
        if ends[e] == ends[e + 1]:
            continue
        av, wv = value(a[i], sa[i], "row"), value(w[e], sw[e], "tile")
        if not back:
            wv = wv.t()
        within(out[i], av @ wv, av.abs() @ wv.abs(), inner, dtype, f"expert {e}")
    return out


ROWS = [
    # counts, n, K
    ([1], 16, 16), ([1], 64, 128), ([1], 2048, 1024), ([3], 272, 4096), ([128], 256, 256),
    ([129], 144, 400), ([300], 1040, 2064), ([1000], 512, 1040), ([4096], 256, 128),
    ([1, 0, 5, 130, 0], 272, 144), ([0, 0, 7], 64, 512), ([256, 256], 256, 384),
    ([127, 1, 128, 513, 0, 33, 700], 528, 656), ([2] * 40, 400, 272), ([0, 0], 64, 64),
    ([900, 40, 0, 1200], 1296, 144),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("counts,n,K", ROWS)
def test_product_and_rows_gradient(lib, counts, n, K, back):
    for k, dtype in enumerate((torch.bfloat16, torch.float32, torch.float16)):
        run_rows(lib, counts, n, K, dtype, back, tail=5 * k, lead=3 * k, seed=k)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("pad", [2, 16, 24])
def test_strided_output(lib, back, pad):
    for dtype in (torch.bfloat16, torch.float32):
        run_rows(lib, [130, 1, 77], 272, 144, dtype, back, pad=pad)
        run_rows(lib, [40], 64, 1024, dtype, back, pad=pad)           # split


def run_dw(lib, counts, n, K, dtype, accumulate=False, tail=0, seed=0, whole=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    ends = segments(counts, 128)
    if whole:
        ends[-1] = ends[-2] + counts[-1]             # the last segment ends with the matrix
    N = ends[-1] + tail
    dy, sy = made((N, n), "col", g)
    x, sx = made((N, K), "col", g, 1e-3)
    for e, c in enumerate(counts):                   # rows that pad a segment are zeros
        dy.view(torch.uint8)[ends[e] + c:ends[e + 1]] = 0
        x.view(torch.uint8)[ends[e] + c:ends[e + 1]] = 0
    if tail:
        for t in (dy, x):
            t.view(torch.uint8)[ends[-1]:] = 0x7f
        for t in (sy, sx):
            t[ends[-1] // 128:] = float("nan")
    before = torch.randn(E, n, K, device="cuda", generator=g).to(dtype)
    dw = before.clone() if accumulate else torch.full_like(before, float("nan"))
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    ws = lib.workspace(lib.product_fp8_ws_bytes(N, n, K, E))
    ws.fill_(0xff)
    lib.moe_product_fp8_dw(dy, sy, x, sx, dw, ws, offsets=offsets, accumulate=accumulate,
                           flags=lib.MOE_CHECK)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        r = slice(a // 128, blocks(b))
        yv = value(dy[a:b], sy[r], "col").t()
        xv = value(x[a:b], sx[r], "col")
        within(dw[e], yv @ xv, yv.abs() @ xv.abs(), max(b - a, 1), dtype, f"expert {e}",
               before[e].double() if accumulate else None)
        if counts[e] == 0:
            assert torch.equal(dw[e], before[e]) if accumulate else (dw[e] == 0).all()
    return dw


@pytest.mark.parametrize("counts,n,K", [
    ([1], 16, 16), ([128], 128, 256), ([300], 272, 144), ([2000], 64, 64), ([5000], 144, 272),
    ([1, 0, 200, 128], 272, 528), ([0, 0, 5], 400, 64), ([257] * 9, 1040, 656), ([0], 64, 64),
    ([40] * 70, 128, 128)])
def test_weights_gradient(lib, counts, n, K):
    for k, dtype in enumerate((torch.float32, torch.bfloat16, torch.float16)):
        for accumulate in (False, True):
            run_dw(lib, counts, n, K, dtype, accumulate, tail=128 * k, seed=k)
    if counts[-1]:
        run_dw(lib, counts, n, K, torch.float32, whole=True)


def test_plain_product_without_offsets(lib):
    g = torch.Generator(device="cuda").manual_seed(1)
    for N, n, K in ((1, 512, 2048), (200, 400, 144), (700, 1040, 528)):
        x, sx = made((N, K), "row", g)
        w, sw = made((n, K), "tile", g)
        dy, sy = made((N, n), "row", g)
        ws = lib.workspace(lib.product_fp8_ws_bytes(N, n, K))
        out, dx = torch.empty(N, n, device="cuda"), torch.empty(N, K, device="cuda")
        lib.moe_product_fp8(x, sx, w, sw, out, ws)
        lib.moe_product_fp8_dx(dy, sy, w, sw, dx, ws)
        xv, wv, yv = value(x, sx, "row"), value(w, sw, "tile"), value(dy, sy, "row")
        within(out, xv @ wv.t(), xv.abs() @ wv.abs().t(), K, torch.float32, "out")
        within(dx, yv @ wv, yv.abs() @ wv.abs(), n, torch.float32, "dx")
        yc, syc = made((N, n), "col", g)
        xc, sxc = made((N, K), "col", g)
        dw = torch.empty(n, K, device="cuda")
        lib.moe_product_fp8_dw(yc, syc, xc, sxc, dw, ws)
        yv, xv = value(yc, syc, "col").t(), value(xc, sxc, "col")
        within(dw, yv @ xv, yv.abs() @ xv.abs(), N, torch.float32, "dw")


def test_no_rows(lib):
    x, sx = torch.empty(0, 64, dtype=E4M3, device="cuda"), torch.empty(0, 1, device="cuda")
    w, sw = made((2, 32, 64), "tile", torch.Generator(device="cuda").manual_seed(1))
    ws = lib.workspace(lib.product_fp8_ws_bytes(0, 32, 64, 2))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    lib.moe_product_fp8(x, sx, w, sw, torch.empty(0, 32, device="cuda"), ws, offsets=off)
    dw = torch.full((2, 32, 64), 3.0, device="cuda")
    dy = torch.empty(0, 32, dtype=E4M3, device="cuda")
    none_y, none_x = torch.empty(0, 32, device="cuda"), torch.empty(0, 64, device="cuda")
    lib.moe_product_fp8_dw(dy, none_y, x, none_x, dw, ws, offsets=off, accumulate=True)
    assert (dw == 3.0).all()
    lib.moe_product_fp8_dw(dy, none_y, x, none_x, dw, ws, offsets=off)
    assert (dw == 0.0).all()


def test_nan_stays_in_its_row_and_expert(lib):
    g = torch.Generator(device="cuda").manual_seed(2)
    counts, n, K = [130, 70, 200], 272, 400
    ends = segments(counts)
    x, sx = made((400, K), "row", g)
    w, sw = made((3, n, K), "tile", g)
    x.view(torch.uint8)[140, 3] = 0x7f
    w.view(torch.uint8)[2, 5, 390] = 0x7f
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    ws = lib.workspace(lib.product_fp8_ws_bytes(400, n, K, 3))
    out, dx = torch.empty(400, n, device="cuda"), torch.empty(400, K, device="cuda")
    lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[140] = True
    want[200:, 5] = True
    assert torch.equal(nan, want)
    dy, sy = made((400, n), "row", g)
    lib.moe_product_fp8_dx(dy, sy, w, sw, dx, ws, offsets=off)
    want = torch.zeros(400, K, dtype=torch.bool, device="cuda")
    want[200:, 390] = True
    assert torch.equal(torch.isnan(dx), want)


@pytest.mark.parametrize("bad", [[0, 5, 3, 20], [0, 5, 21, 21], [-1, 5, 6, 7], [0, 30, 10, 20],
                                 [2, 1, 1, 1]])
def test_offsets_that_are_not_valid(lib, bad):
    """Reported, and nothing is written."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N, n, K, E = 20, 64, 512, 3
    x, sx = made((N, K), "row", g)
    w, sw = made((E, n, K), "tile", g)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    ws = lib.workspace(lib.product_fp8_ws_bytes(N, n, K, E))
    out = torch.full((N, n), -7.0, device="cuda")
    with pytest.raises(lib.MoeError):
        lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off, flags=lib.MOE_CHECK)
    lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off)
    assert (out == -7.0).all()


@pytest.mark.parametrize("bad", [[0, 100, 256], [0, 128, 200], [128, 0, 256], [0, 128, 512]])
def test_weights_gradient_offsets_that_are_not_valid(lib, bad):
    g = torch.Generator(device="cuda").manual_seed(2)
    N, n, K, E = 256, 64, 64, 2
    dy, sy = made((N, n), "col", g)
    x, sx = made((N, K), "col", g)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    ws = lib.workspace(lib.product_fp8_ws_bytes(N, n, K, E))
    dw = torch.full((E, n, K), -7.0, device="cuda")
    with pytest.raises(lib.MoeError):
        lib.moe_product_fp8_dw(dy, sy, x, sx, dw, ws, offsets=off, flags=lib.MOE_CHECK)
    assert (dw == -7.0).all()


def test_same_bits_again_on_a_stream_and_in_a_graph(lib):
    g = torch.Generator(device="cuda").manual_seed(3)
    counts, n, K = [300, 0, 130], 528, 400
    N = 430
    x, sx = made((N, K), "row", g)
    w, sw = made((3, n, K), "tile", g)
    off = torch.tensor(segments(counts), dtype=torch.int32, device="cuda")
    ws = lib.workspace(lib.product_fp8_ws_bytes(N, n, K, 3))
    out = torch.empty(N, n, device="cuda")
    lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off)
    first = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off)
    off.copy_(torch.tensor([0, 100, 430, 430], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    lib.moe_product_fp8(x, sx, w, sw, out, ws, offsets=off)
    assert torch.equal(out, replayed) and not torch.equal(out, first)
