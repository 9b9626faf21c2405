"""GPU: E4M3 codes and scales by row, by column and by tile, bit for bit against the definition on
the CPU (fp32 quotients by IEEE division, rounded to nearest even)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def reference(x, bn, bk):
    """Codes (as bits) and scales of a CPU matrix in blocks of bn x bk."""
    n, K = x.shape
    x = x.float()
    N, C = -(-n // bn) * bn, -(-K // bk) * bk
    full = torch.zeros(N, C)
    full[:n, :K] = x
    parts = full.view(N // bn, bn, C // bk, bk)
    scale = torch.nan_to_num(parts.abs(), nan=0.0, posinf=float("inf")).amax((1, 3)) / 448.0
    s = scale[:, None, :, None]
    q = torch.where(s > 0, parts / s, torch.where(parts.isnan(), parts, 0.0))
    codes = q.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8).view(N, C)[:n, :K]
    return codes, scale


def same_codes(got, ref, name):
    """Equal codes; a zero's sign does not count."""
    got, ref = got.cpu().view(torch.uint8).int(), ref.int()
    got, ref = (torch.where(c == 0x80, 0, c) for c in (got, ref))
    got, ref = (torch.where((c & 0x7f) == 0x7f, 0x7f, c) for c in (got, ref))   # one NaN
    assert torch.equal(got, ref), f"{name}: {(got != ref).sum()} codes differ"


def check_rows(lib, x, dtype_codes=E4M3):
    N, K = x.shape
    b = lib.fp8_blocks
    mk = dict(device="cuda")
    codes, col_codes = (torch.full((N, K), 99, dtype=torch.uint8, **mk).view(dtype_codes) for _ in "ab")
    scales = torch.full((N, b(K)), float("nan"), **mk)
    col_scales = torch.full((b(N), K), float("nan"), **mk)
    host = x.cpu()
    rc, rs = reference(host, 1, 128)
    cc, cs = reference(host, 128, 1)

    def compare(what):
        if "r" in what:
            assert torch.equal(scales.cpu(), rs), what
            same_codes(codes, rc, what)
        if "c" in what:
            assert torch.equal(col_scales.cpu(), cs), what
            same_codes(col_codes, cc, what)

    lib.moe_quantize_fp8(x, codes, scales, col_codes, col_scales)
    compare("rc")
    for what in "rc":
        for t in (codes, col_codes):
            t.view(torch.uint8).fill_(99)
        for t in (scales, col_scales):
            t.fill_(float("nan"))
        if what == "r":
            lib.moe_quantize_fp8(x, codes, scales)
            assert torch.isnan(col_scales).all()
        else:
            lib.moe_quantize_fp8(x, col_codes=col_codes, col_scales=col_scales)
            assert torch.isnan(scales).all()
        compare(what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N,K", [(1, 16), (1, 7168), (127, 128), (128, 144), (129, 1040),
                                 (300, 2064), (1025, 64)])
def test_rows_and_columns(lib, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    x = torch.randn(N, K, device="cuda", generator=g)
    x *= torch.exp2(torch.randint(-12, 5, (N, 1), device="cuda", generator=g))
    x[:, K // 2] = 0.0
    check_rows(lib, x.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("E,n,K", [(1, 16, 16), (3, 130, 272), (2, 1408, 2064), (5, 128, 128),
                                   (1, 7, 48)])
def test_tiles(lib, E, n, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + K)
    w = (torch.randn(E, n, K, device="cuda", generator=g) * 0.02).to(dtype)
    w[0, :n // 2] *= 100
    codes = torch.empty(E, n, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, lib.fp8_blocks(n), lib.fp8_blocks(K), device="cuda")
    lib.moe_quantize_fp8_tiles(w, codes, scales)
    for e in range(E):
        rc, rs = reference(w[e].cpu(), 128, 128)
        assert torch.equal(scales[e].cpu(), rs)
        same_codes(codes[e], rc, f"expert {e}")


def test_every_bf16_under_many_scales(lib):
    """Each positive and negative bf16 value as a neighbour of every kind of largest value, among
    them scales where the quotient is divided and ones below the normal range."""
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    every = every[torch.isfinite(every)]
    tops = [1.0, 1.0078125, 1.75, 448.0, 3.3e38, 2.0 ** -60, 2.0 ** -70, 1e-38, 2.0 ** 70, 0.0299]
    rows = []
    for top in tops:
        v = every[every.abs() <= top]
        v = torch.cat([v, torch.zeros(-v.numel() % 127)])
        block = torch.full((v.numel() // 127, 128), top)
        block[:, 1:] = v.view(-1, 127)
        rows.append(block)
    x = torch.cat(rows).bfloat16()
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[0], 1, device="cuda")
    lib.moe_quantize_fp8(x.cuda(), codes, scales)
    rc, rs = reference(x, 1, 128)
    assert torch.equal(scales.cpu(), rs)
    same_codes(codes, rc, "every bf16")


def test_random_fp32_quotients(lib):
    """fp32 values next to the borders between two codes: quotients that differ by units of 2^-24."""
    g = torch.Generator().manual_seed(3)
    top = torch.rand(20000, 1, generator=g) + 0.5
    scale = top / 448.0
    odd = torch.randint(8, 240, (20000, 127), generator=g) * 2 + 1     # halves of the code's steps
    border = odd.float() / 16.0 * torch.exp2(torch.randint(-6, 4, (20000, 127), generator=g))
    v = (border * scale).clamp(max=top)
    step = torch.randint(-2, 3, v.shape, generator=g, dtype=torch.int32)
    v = (v.view(torch.int32) + step).view(torch.float32).minimum(top)
    x = torch.cat([top, v], 1)
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[0], 1, device="cuda")
    lib.moe_quantize_fp8(x.cuda(), codes, scales)
    rc, rs = reference(x, 1, 128)
    assert torch.equal(scales.cpu(), rs)
    same_codes(codes, rc, "borders")


def test_nan_and_infinity(lib):
    x = torch.randn(256, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[5, 7] = float("nan")
    x[9, 130] = float("inf")
    x[11, 131] = -float("inf")
    x[130:, 3] = 0.0
    x[140, 3] = float("nan")             # alone in a block of zeros
    check_rows(lib, x)
    check_rows(lib, x.bfloat16())


def test_strides_and_offsets(lib):
    g = torch.Generator(device="cuda").manual_seed(6)
    wide = torch.randn(200, 512, device="cuda", generator=g)
    for dtype in (torch.float32, torch.bfloat16):
        w = wide.to(dtype)
        for cut in (w[:, :256], w[:, 8:264], w[1:, 1:257], w[3:, 5:133], w[::2, :128]):
            check_rows(lib, cut)


def test_rows_are_those_of_the_fp8_dispatch(lib):
    T, d, E, R = 130, 256, 8, 2
    x = torch.randn(T, d, device="cuda").bfloat16()
    idx = torch.randint(0, E, (T, 1), device="cuda").int().repeat(1, R)
    idx[:, 1] = (idx[:, 0] + 1) % E
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = [torch.empty(k, **i32) for k in (E, E + 1, T * R, T * R)]
    xq = torch.empty(T * R, d, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T * R, d // 128, device="cuda")
    lib.moe_dispatch_fp8(x, idx, E, *plan, xq, xs, lib.workspace(lib.dispatch_ws_bytes(T, d, E, R)))
    rows = x[(plan[2] // R).long()]
    codes, scales = torch.empty_like(xq), torch.empty_like(xs)
    lib.moe_quantize_fp8(rows, codes, scales)
    assert torch.equal(scales, xs)
    same_codes(codes, xq.cpu(), "dispatch")


def test_more_rows_than_32_bits_of_elements(lib):
    """2^32 elements and more: rows behind the 32-bit offset are where they belong."""
    N, K = (1 << 18) + 129, 1 << 14
    x = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    x[-130:] = torch.randn(130, K, device="cuda").bfloat16()
    codes = torch.empty(N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, K // 128, device="cuda")
    col_codes, col_scales = torch.empty_like(codes), torch.empty(lib.fp8_blocks(N), K, device="cuda")
    lib.moe_quantize_fp8(x, codes, scales, col_codes, col_scales)
    tail = x[-257:].cpu()                # whole blocks of columns: N - 257 is a multiple of 128
    assert (N - 257) % 128 == 0
    rc, rs = reference(tail, 1, 128)
    cc, cs = reference(tail, 128, 1)
    assert torch.equal(scales[-257:].cpu(), rs) and torch.equal(col_scales[-3:].cpu(), cs)
    same_codes(codes[-257:], rc, "rows")
    same_codes(col_codes[-257:], cc, "columns")
    assert not codes[:1000].any() and not scales[:1000].any()
