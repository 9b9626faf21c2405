"""GPU: gradient norm and AdamW step against 64-bit computations.

Bounds of the fp32 step, with e = 2^-24: m within 3 e (|beta1 m| + |c1 g'|), v
within 4 e v; the update m s / (sqrt(v) r + eps) within its share of m's error
plus 8 e of itself; p within 3 e (|p| + |update|) more, then the store's rounding.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.98, eps=1e-8, step=3, seed=11)


def tensor(n, p16, g16, bits, master, shift, seed, zeros=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(scale):
        return torch.randn(n + shift, generator=gen, device="cuda").mul_(scale)[shift:]

    t = {"p": randn(0.1), "g": randn(0.03)}
    if p16:
        base = torch.empty(n + shift, dtype=torch.bfloat16, device="cuda")[shift:]
        t["master"] = t["p"].clone() if master else None
        t["p"] = base.copy_(t["p"])
    if g16:
        base = torch.empty(n + shift, dtype=torch.bfloat16, device="cuda")[shift:]
        t["g"] = base.copy_(t["g"])
    if bits == 32:
        t["m"], t["v"] = randn(0.01), randn(0.02).square_()
        if zeros:
            t["m"].zero_(), t["v"].zero_()
    else:
        blocks = -(-n // 256)
        for name in ("m", "v"):
            codes = randn(100.0).clamp_(-448, 448)
            codes = (codes.abs() if name == "v" else codes).to(torch.float8_e4m3fn)
            base = torch.empty(n + shift, dtype=torch.float8_e4m3fn, device="cuda")[shift:]
            t[name] = base.copy_(codes)
            t[name + "_scale"] = torch.rand(blocks, generator=gen, device="cuda") * 5e-5
            if zeros:
                t[name].view(torch.uint8).zero_()
                t[name + "_scale"].zero_()
    return t


def values(t, name):
    x = t[name].double()
    if name + "_scale" in t:
        x = x * t[name + "_scale"].double().repeat_interleave(256)[:x.numel()]
        x = x * x if name == "v" else x
    return x


def expected(t, wd, coef=1.0, h=HYPER):
    """The step's results and bounds in float64, from copies of the inputs."""
    f = lambda v: float(np.float32(v))  # noqa: E731
    b1, b2, c1, c2 = f(h["beta1"]), f(h["beta2"]), f(1 - h["beta1"]), f(1 - h["beta2"])
    g = t["g"].double() * coef
    m0, v0 = values(t, "m"), values(t, "v")
    m, v = b1 * m0 + c1 * g, b2 * v0 + c2 * g * g
    m_err = 5 * EPS * ((b1 * m0).abs() + (c1 * g).abs())
    p0 = (t["master"] if t.get("master") is not None else t["p"]).double()
    s = f(h["lr"] / (1 - h["beta1"] ** h["step"]))
    r = f(1 / math.sqrt(1 - h["beta2"] ** h["step"]))
    denom = v.sqrt() * r + f(h["eps"])
    upd = m * s / denom
    p = p0 * f(1 - h["lr"] * wd) - upd
    p_err = m_err * s / denom + 10 * EPS * upd.abs() + 4 * EPS * (p0.abs() + upd.abs())
    return dict(m=m, v=v, p=p, m_err=m_err, v_err=6 * EPS * v + 1e-44, p_err=p_err)


def make(lib, t, wd):
    return lib.AdamWTensor(t["p"], t["g"], t["m"], t["v"], master=t.get("master"),
                           m_scale=t.get("m_scale"), v_scale=t.get("v_scale"), weight_decay=wd)


def check(t, want, name):
    p_err = want["p_err"]
    if t.get("master") is not None:
        assert ((t["master"].double() - want["p"]).abs() <= p_err).all(), name
    stored = p_err + (2.0 ** -8 * (want["p"].abs() + p_err) if t["p"].dtype == torch.bfloat16 else 0)
    assert ((t["p"].double() - want["p"]).abs() <= stored + 1e-40).all(), name
    if "m_scale" not in t:
        assert ((t["m"].double() - want["m"]).abs() <= want["m_err"] + 1e-44).all(), name
        assert ((t["v"].double() - want["v"]).abs() <= want["v_err"]).all(), name
        return
    n = t["m"].numel()
    for key, exact, err in (("m", want["m"], want["m_err"]),
                            ("v", want["v"].sqrt(), 4 * EPS * want["v"].sqrt())):
        scales = t[key + "_scale"].double()
        full = torch.zeros(scales.numel() * 256, dtype=torch.float64, device="cuda")
        full[:n] = exact.abs()
        top = full.view(-1, 256).amax(1) / 448
        slack = torch.zeros_like(full)
        slack[:n] = err
        slack = slack.view(-1, 256).amax(1) / 448
        assert ((scales - top).abs() <= slack + 2 * EPS * top + 1e-38).all(), f"{name} {key}_scale"
        unit = scales.repeat_interleave(256)[:n]
        got = t[key].double() * unit
        # the neighbours of r are at most r / 8 apart (2^-9 below 2^-6)
        spacing = torch.maximum(exact.abs() / 8, unit * 2.0 ** -9) + 2 * err + 1e-6 * exact.abs()
        assert ((got - exact).abs() <= spacing + 1e-38).all(), f"{name} {key}"
        if key == "v":
            assert ((got > 0) | (exact < 1e-37) | (unit == 0)).all(), f"{name}: a root went to zero"


SIZES = [1, 7, 255, 256, 257, 2048, 5000, 70001]
KINDS = [  # p16, g16, bits, master
    (True, False, 32, False), (True, True, 32, True), (False, False, 32, False),
    (False, True, 8, False), (True, False, 8, False), (True, True, 8, True)]


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("kind", KINDS)
def test_step(lib, kind, shift):
    p16, g16, bits, master = kind
    ts = [tensor(n, p16, g16, bits, master, shift, seed=n) for n in SIZES]
    wds = [0.0 if n < 300 else 0.1 for n in SIZES]
    want = [expected(t, wd) for t, wd in zip(ts, wds)]
    grads = [t["g"].clone() for t in ts]
    lib.moe_adamw_step(lib.AdamWList([make(lib, t, wd) for t, wd in zip(ts, wds)]), **HYPER)
    for n, t, w, g in zip(SIZES, ts, want, grads):
        check(t, w, f"n={n}")
        assert torch.equal(t["g"], g)


@pytest.mark.parametrize("bits", [8, 32])
def test_first_step_and_zero_gradients(lib, bits):
    """From zero states; where the gradient is zero nothing but the decay moves p."""
    t = tensor(3000, False, False, bits, False, 0, seed=1, zeros=True)
    t["g"][:700] = 0
    h = dict(HYPER, step=1)
    want = expected(t, 0.1, h=h)
    p0 = t["p"].clone()
    lib.moe_adamw_step(lib.AdamWList([make(lib, t, 0.1)]), **h)
    check(t, want, "first step")
    assert torch.allclose(t["p"][:700], p0[:700] * (1 - 1e-3), rtol=2e-7, atol=0)
    assert (values(t, "m")[:700] == 0).all() and (values(t, "v")[:700] == 0).all()


def test_many_tensors(lib):
    """More tensors than one launch takes, empty ones and mixed kinds among them."""
    ts, wds = [], []
    for k in range(700):
        p16, g16, bits, master = KINDS[k % len(KINDS)]
        ts.append(tensor((k * 37) % 900, p16, g16, bits, master, k % 3, seed=k))
        wds.append(0.01 * (k % 5))
    want = [expected(t, wd) for t, wd in zip(ts, wds)]
    items = lib.AdamWList([make(lib, t, wd) for t, wd in zip(ts, wds)])
    norm = torch.empty(4, device="cuda")
    lib.moe_grad_norm(items, 0.0, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    total = math.sqrt(sum(float(t["g"].double().square().sum()) for t in ts))
    assert abs(float(norm[0]) - total) <= 1e-6 * total and norm[1:].tolist() == [1.0, 1.0, 0.0]
    lib.moe_adamw_step(items, norm=norm, **HYPER)
    for k, (t, w) in enumerate(zip(ts, want)):
        check(t, w, f"tensor {k}")


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("bits", [8, 32])
def test_clip(lib, bits, max_norm):
    ts = [tensor(n, True, n % 2 == 0, bits, False, 0, seed=n) for n in (100, 5001, 300000)]
    items = lib.AdamWList([make(lib, t, 0.0) for t in ts])
    norm = torch.empty(4, device="cuda")
    lib.moe_grad_norm(items, max_norm, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    total = math.sqrt(sum(float(t["g"].double().square().sum()) for t in ts))
    coef = min(1.0, max_norm / (total + 1e-6)) if max_norm > 0 else 1.0
    # squares of 8 values in fp32: 8 e of the sum, half that of its root, and the roundings
    assert abs(float(norm[0]) - total) <= 8 * EPS * total
    assert abs(float(norm[1]) - coef) <= 12 * EPS * coef
    want = [expected(t, 0.0, coef=float(norm[1])) for t in ts]
    lib.moe_adamw_step(items, norm=norm, **HYPER)
    for t, w in zip(ts, want):
        check(t, w, "clipped")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_gradients_that_are_not_finite_skip_the_step(lib, bad):
    ts = [tensor(n, True, False, 8, False, 0, seed=n) for n in (100, 50000)]
    ts[1]["g"][49999] = bad
    items = lib.AdamWList([make(lib, t, 0.1) for t in ts])
    norm = torch.empty(4, device="cuda")
    lib.moe_grad_norm(items, 1.0, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    assert float(norm[2]) == 0.0
    before = [{k: v.clone() for k, v in t.items() if v is not None} for t in ts]
    lib.moe_adamw_step(items, norm=norm, **HYPER)
    for a, b in zip(ts, before):
        for k, v in b.items():
            assert torch.equal(a[k].view(torch.uint8), v.view(torch.uint8)), k


def test_empty_list(lib):
    items = lib.AdamWList([])
    norm = torch.full((4,), 9.0, device="cuda")
    lib.moe_grad_norm(items, 1.0, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    assert norm.tolist() == [0.0, 1.0, 1.0, 0.0]
    lib.moe_adamw_step(items, norm=norm, **HYPER)


def test_eight_bit_rounding_is_fair(lib):
    """Over many seeds the stored states average to the exact ones: with k seeds the mean of
    an error in (-s, s) of variance <= s^2 / 4 (s the spacing) is within 6 s / (2 sqrt k), and
    the mean over the n elements of error / spacing within 6 / (2 sqrt(k n / 16)) (dithers of
    neighbours in a hash are taken as dependent)."""
    n, k = 4096, 64
    start = tensor(n, False, False, 8, False, 0, seed=5)
    want = expected(start, 0.0)
    for key, exact in (("m", want["m"]), ("v", want["v"].sqrt())):
        total = torch.zeros(n, dtype=torch.float64, device="cuda")
        for seed in range(k):
            t = {a: b.clone() for a, b in start.items() if b is not None}
            lib.moe_adamw_step(lib.AdamWList([make(lib, t, 0.0)]), **dict(HYPER, seed=seed))
            unit = t[key + "_scale"].double().repeat_interleave(256)
            total += t[key].double() * unit - exact
        r = exact.abs() / unit
        spacing = torch.maximum(torch.exp2(torch.floor(torch.log2(r.clamp_min(2.0 ** -6)))) / 8,
                                torch.tensor(2.0 ** -9, dtype=torch.float64)) * unit
        top = r < 440            # values at the top of the range only round down
        mean = total / k / spacing
        assert float(mean[top].abs().max()) <= 6 / (2 * math.sqrt(k)), key
        assert abs(float(mean[top].mean())) <= 6 / (2 * math.sqrt(k * n / 16)), key


def test_eight_bit_state_follows(lib):
    """With a constant gradient sqrt(v) grows towards |g| as it does in 64 bits, although one
    step moves it by far less than a code's spacing."""
    n, steps = 2048, 150
    t = tensor(n, False, False, 8, False, 0, seed=3, zeros=True)
    t["g"].copy_(torch.linspace(0.5, 1.0, n, device="cuda"))
    h = dict(HYPER, beta2=0.999, lr=1e-4)
    items = lib.AdamWList([make(lib, t, 0.0)])
    for step in range(1, steps + 1):
        lib.moe_adamw_step(items, **dict(h, step=step, seed=step))
    exact = t["g"].double() * math.sqrt(1 - 0.999 ** steps)
    ratio = values(t, "v").sqrt() / exact
    assert 0.97 < float(ratio.mean()) < 1.03
    assert 0.95 < float((values(t, "m") / t["g"].double()).mean()) < 1.05


@pytest.mark.parametrize("bits", [8, 32])
def test_same_bits_every_time_and_in_a_graph(lib, bits):
    outs = []
    for captured in (False, False, True):
        ts = [tensor(n, True, False, bits, True, 0, seed=n) for n in (3, 4096, 100003)]
        items = lib.AdamWList([make(lib, t, 0.1) for t in ts])
        norm = torch.empty(4, device="cuda")
        ws = lib.workspace(lib.grad_norm_ws_bytes(items))

        def step():
            lib.moe_grad_norm(items, 0.1, norm, ws)
            lib.moe_adamw_step(items, norm=norm, **HYPER)

        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        outs.append([v.view(torch.uint8) for t in ts for v in t.values()])
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def mix(x):
    x = (x ^ (x >> np.uint64(16))) * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF)
    x = (x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def stored_on_the_host(x, scale, dither, least):
    """Codes of x (fp32) by the definition: scale, quotient and rounding operation by operation."""
    f = np.float32
    inv = np.where(scale >= f(2.0 ** -126), f(1) / np.maximum(scale, f(2.0 ** -126)), f(0))
    r = np.minimum(np.abs(x) * np.repeat(inv, 256)[:x.size], f(448))
    shift = np.where(r < f(2.0 ** -6), f(2.0 ** -6), f(0))
    kept = ((r + shift).view(np.uint32) + dither) & np.uint32(0xFFF00000)
    q = np.where(r > 0, np.clip(kept.view(np.float32) - shift, f(least), f(448)), f(0))
    return np.copysign(q, x)


@pytest.mark.parametrize("n,shift", [(1000, 0), (4096, 0), (40000, 0), (40000, 3)])
def test_eight_bit_states_bit_for_bit(lib, n, shift):
    """Codes and scales after three steps equal those of the formulas, computed on the host one
    fp32 operation at a time, bit for bit."""
    f = np.float32
    t = tensor(n, True, False, 8, False, shift, seed=n)
    h = dict(HYPER)
    f32 = lambda a: a.float().cpu().numpy()  # noqa: E731
    m8, v8, ms, vs = f32(t["m"]), f32(t["v"]), f32(t["m_scale"]), f32(t["v_scale"])
    g = f32(t["g"])
    other = tensor(700, True, False, 8, False, 0, seed=1)        # its place in the list is 0
    items = lib.AdamWList([make(lib, other, 0.0), make(lib, t, 0.1)])
    b1, b2 = f(h["beta1"]), f(h["beta2"])
    c1, c2 = f(1 - h["beta1"]), f(1 - h["beta2"])
    for step in range(1, 4):
        h.update(step=step, seed=70 + step)
        lib.moe_adamw_step(items, **h)
        place = mix(np.uint64((h["seed"] + 0x9E3779B1) & 0xFFFFFFFF))
        pair = np.arange((n + 1) // 2, dtype=np.uint64)
        bits = mix((pair * np.uint64(0x9E3779B1) + place) & np.uint64(0xFFFFFFFF))
        half = np.stack([bits & np.uint64(0xFFFF), bits >> np.uint64(16)], 1).reshape(-1)[:n]
        dither = (half * np.uint64(16) + np.uint64(8)).astype(np.uint32)
        m = m8 * np.repeat(ms, 256)[:n] * b1 + g * c1
        q = v8 * np.repeat(vs, 256)[:n]
        u = np.sqrt(q * q * b2 + g * g * c2)
        full = np.zeros((ms.size * 256, 2), f)
        full[:n, 0], full[:n, 1] = np.abs(m), u
        top = full.reshape(-1, 256, 2).max(1) * (f(1) / f(448))
        ms, vs = (np.where(top[:, k] >= f(2.0 ** -126), top[:, k], f(0)) for k in (0, 1))
        m8 = stored_on_the_host(m, ms, dither, 0.0)
        v8 = stored_on_the_host(u, vs, dither, 2.0 ** -9)
        for name, want in (("m", m8), ("v", v8), ("m_scale", ms), ("v_scale", vs)):
            got = f32(t[name])
            assert np.array_equal(got, want), f"step {step} {name}: {(got != want).sum()} differ"


def test_tensor_past_32_bit_offsets(lib):
    """More than 2^31 elements: the step and the norm reach the end."""
    n = 2 ** 31 + 1024
    dev = dict(device="cuda")
    t = {"p": torch.zeros(n, dtype=torch.bfloat16, **dev), "g": torch.zeros(n, dtype=torch.bfloat16, **dev),
         "m": torch.zeros(n, dtype=torch.float8_e4m3fn, **dev), "v": torch.zeros(n, dtype=torch.float8_e4m3fn, **dev),
         "m_scale": torch.zeros(n // 256, **dev), "v_scale": torch.zeros(n // 256, **dev)}
    t["p"][-512:] = torch.randn(512, **dev).bfloat16()
    t["g"][-512:] = torch.randn(512, **dev).bfloat16()
    last = {k: (x[-512:] if x.numel() == n else x[-2:]) for k, x in t.items()}
    items = lib.AdamWList([make(lib, t, 0.1)])
    norm = torch.empty(4, **dev)
    lib.moe_grad_norm(items, 0.0, norm, lib.workspace(lib.grad_norm_ws_bytes(items)))
    total = float(last["g"].double().square().sum().sqrt())
    assert abs(float(norm[0]) - total) <= 8 * EPS * total
    want = expected(last, 0.1)
    lib.moe_adamw_step(items, **HYPER)
    check(last, want, "the end")
    for name in ("p", "m", "v"):
        for part in t[name].view(torch.int16 if name == "p" else torch.uint8)[:-512].split(2 ** 29):
            assert not part.any(), name
