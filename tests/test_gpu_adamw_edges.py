"""GPU: the optimiser step and the norm at the ends of their ranges and over long lists.  Helpers and
bounds are those of test_gpu_adamw."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_adamw import (EPS, HYPER, KINDS, check, expected, make, mix, stored_on_the_host,
                                  tensor)

pytestmark = pytest.mark.gpu


def dithers(n, place, seed):
    """The dither of n elements of the place-th tensor, by its definition."""
    golden, low = np.uint64(0x9E3779B1), np.uint64(0xFFFFFFFF)
    start = mix(np.uint64((seed + place * 0x9E3779B1) & 0xFFFFFFFF))
    bits = mix((np.arange((n + 1) // 2, dtype=np.uint64) * golden + start) & low)
    half = np.stack([bits & np.uint64(0xFFFF), bits >> np.uint64(16)], 1).reshape(-1)[:n]
    return (half * np.uint64(16) + np.uint64(8)).astype(np.uint32)


# whole chunks; a chunk that ends early, its whole blocks and its last one; unaligned
@pytest.mark.parametrize("n,shift", [(4096, 0), (2048 + 700, 0), (4096, 3)])
def test_small_roots_beside_large_ones(lib, n, shift):
    """sqrt(v) > 0 gets a code above 0 however small it is beside its block's largest: gradients of
    1 and of 1e-13 .. 1e-6 from zero states, codes and scales bit for bit."""
    f = np.float32
    t = tensor(n, False, False, 8, False, shift, seed=n, zeros=True)
    gen = torch.Generator(device="cuda").manual_seed(7)
    small = torch.rand(n, generator=gen, device="cuda") < 0.7
    power = torch.rand(n, generator=gen, device="cuda") * 7 - 13
    sign = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    t["g"].copy_(torch.where(small, 10.0 ** power, 1.0) * sign)
    t["g"][5::97] = 0
    h = dict(HYPER, step=1)
    lib.moe_adamw_step(lib.AdamWList([make(lib, t, 0.0)]), **h)
    f32 = lambda a: a.float().cpu().numpy()  # noqa: E731
    g = f32(t["g"])
    m, u = g * f(1 - h["beta1"]), np.sqrt(g * g * f(1 - h["beta2"]))
    blocks = -(-n // 256)
    for name, x, least in (("m", m, 0.0), ("v", u, 2.0 ** -9)):
        full = np.zeros(blocks * 256, f)
        full[:n] = np.abs(x)
        scale = full.reshape(-1, 256).max(1) * (f(1) / f(448))
        want = stored_on_the_host(x, scale, dithers(n, 0, h["seed"]), least)
        got = f32(t[name])
        assert np.array_equal(f32(t[name + "_scale"]), scale), name
        assert np.array_equal(got, want), f"{name}: {(got != want).sum()} differ"
    assert ((f32(t["v"]) > 0) == (g != 0)).all()


def norm_of(lib, grads, max_norm):
    """The record of moe_grad_norm over fp32 gradients."""
    items = lib.AdamWList([lib.AdamWTensor(g, g, g, g) for g in grads])
    norm = torch.full((4,), 9.0, device="cuda")
    lib.moe_grad_norm(items, max_norm, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    return norm.tolist()


@pytest.mark.parametrize("max_norm", [1e-46, 1e-60, 5e-324])
def test_limit_below_the_smallest_fp32_number(lib, max_norm):
    """A limit above zero clips, however small: the factor rounds to 0, it is not 1."""
    g = torch.full((1000,), 0.5, device="cuda")
    norm = norm_of(lib, [g], max_norm)
    assert norm[1:] == [0.0, 1.0, 0.0]


@pytest.mark.parametrize("n", [40, 70001])
@pytest.mark.parametrize("max_norm", [0.0, 2.0, 1e300, float("inf")])
def test_record_of_norms_that_are_not_finite(lib, n, max_norm):
    """An infinite gradient or a sum of squares above the fp32 range: norm inf, factor 0; a NaN: both
    NaN.  Without a limit the factor is 1."""
    inf, nan = float("inf"), float("nan")
    for values, want in (((inf,), inf), ((-inf, 3.0), inf), ((1e25,), inf), ((1.5e19, 1.5e19), inf),
                         ((nan,), nan), ((inf, nan), nan), ((nan, inf), nan)):
        g = torch.full((n,), 0.01, device="cuda")
        for k, value in enumerate(values):
            g[(n - 1) // (k + 1)] = value
        norm = norm_of(lib, [torch.ones(300, device="cuda"), g], max_norm)
        factor = 1.0 if max_norm == 0 else 0.0 if want == inf else nan
        assert np.array_equal(norm, [want, factor, 0.0, 0.0], equal_nan=True), (values, norm)


def test_launches_are_counted(lib):
    """A launch for each kind of state in a run of at most 256 tensors; two of the norm at least."""
    def count(call):
        before = lib.kernel_launches()
        call()
        return lib.kernel_launches() - before

    def items(kinds):
        return lib.AdamWList([make(lib, tensor(n, False, False, bits, False, 0, seed=n), 0.0)
                              for n, bits in kinds])

    norm = torch.empty(4, device="cuda")
    for kinds, steps, norms in (([(100, 32)], 1, 2), ([(100, 8)], 1, 2), ([(100, 8), (7, 32)], 2, 2),
                                ([(10, 32)] * 300, 2, 3), ([], 0, 1)):
        x = items(kinds)
        ws = lib.workspace(lib.grad_norm_ws_bytes(x))
        assert count(lambda: lib.moe_grad_norm(x, 1.0, norm, ws)) == norms
        assert count(lambda: lib.moe_adamw_step(x, norm=norm, **HYPER)) == steps


@pytest.mark.parametrize("bits", [8, 32])
def test_replays_repeat_the_captured_step(lib, bits):
    """lr, step and seed are values of the call: a replay is the same step again, not the next."""
    start = tensor(5000, True, False, bits, True, 0, seed=2)
    results = []
    for captured in (False, True):
        t = {k: v.clone() for k, v in start.items()}
        items = lib.AdamWList([make(lib, t, 0.1)])
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                lib.moe_adamw_step(items, **HYPER)
        for _ in range(3):
            graph.replay() if captured else lib.moe_adamw_step(items, **HYPER)
        torch.cuda.synchronize()
        results.append(t)
    for k in start:
        assert torch.equal(*(t[k].view(torch.uint8) for t in results)), k


# what makes a warp take eight blocks in a row (8-bit states), two (32 bits) and the norm four
LONG = 8 * 2048 * 152 * 8


@pytest.mark.parametrize("kind", KINDS)
def test_long_lists(lib, kind):
    """The longest runs a warp takes, in a list with a ragged and an unaligned tensor: every element."""
    p16, g16, bits, master = kind
    ts = [tensor(n, p16, g16, bits, master, shift, seed=n % 1000)
          for n, shift in ((LONG, 0), (100_003, 0), (70_001, 3))]
    items = lib.AdamWList([make(lib, t, 0.1) for t in ts])
    norm = torch.empty(4, device="cuda")
    lib.moe_grad_norm(items, 1.0, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    total = math.sqrt(sum(float(t["g"].double().square().sum()) for t in ts))
    # squares of 8 values in fp32: 8 e of the sum, half that of its root, and the roundings
    assert abs(float(norm[0]) - total) <= 8 * EPS * total
    want = [expected(t, 0.1, coef=float(norm[1])) for t in ts]
    lib.moe_adamw_step(items, norm=norm, **HYPER)
    for t, w in zip(ts, want):
        check(t, w, f"n={t['p'].numel()}")


def test_long_list_bit_for_bit(lib):
    """Codes and scales of a list whose warps take eight blocks in a row."""
    f = np.float32
    t = tensor(LONG + 300, False, True, 8, False, 0, seed=4)
    h = dict(HYPER)
    f32 = lambda a: a.float().cpu().numpy()  # noqa: E731
    old = {k: f32(t[k]) for k in ("m", "v", "m_scale", "v_scale", "g")}
    lib.moe_adamw_step(lib.AdamWList([make(lib, t, 0.0)]), **h)
    n = t["m"].numel()
    dither = dithers(n, 0, h["seed"])
    g = old["g"]
    m = old["m"] * np.repeat(old["m_scale"], 256)[:n] * f(h["beta1"]) + g * f(1 - h["beta1"])
    q = old["v"] * np.repeat(old["v_scale"], 256)[:n]
    u = np.sqrt(q * q * f(h["beta2"]) + g * g * f(1 - h["beta2"]))
    for name, x, least in (("m", m, 0.0), ("v", u, 2.0 ** -9)):
        full = np.zeros(-(-n // 256) * 256, f)
        full[:n] = np.abs(x)
        scale = full.reshape(-1, 256).max(1) * (f(1) / f(448))
        assert np.array_equal(f32(t[name + "_scale"]), scale), name
        got, want = f32(t[name]), stored_on_the_host(x, scale, dither, least)
        assert np.array_equal(got, want), f"{name}: {(got != want).sum()} differ"
