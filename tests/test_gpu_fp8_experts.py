"""GPU: router, sort, fp8 codes, products and all gradients together, as examples/fp8_experts.py
uses them; each step against 64 bits on the inputs that it got in the chain, and the block's
gradients against those of the block without rounding."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "fp8_experts.py")


def load():
    spec = importlib.util.spec_from_file_location("fp8_experts", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def value(codes, scales, form):
    n, K = codes.shape[-2:]
    v = scales.double()
    if form != "row":
        v = v.repeat_interleave(128, -2)[..., :n, :]
    if form != "col":
        v = v.repeat_interleave(128, -1)[..., :K]
    return codes.double() * v


def close(got, ref, size, k, dtype, name):
    """A product of k terms of total magnitude `size`: 2^-23 (292 + 3 blocks) of it for the sums
    (33 units a 32-deep step of a block, the scales' roundings), then the store's half step."""
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    slack = (292 + 3 * -(-k // 128)) * 2.0 ** -23 * size
    off = (got.double() - ref).abs() - slack - half * (ref.abs() + slack) - 2.0 ** -134
    assert float(off.max()) <= 0, f"{name}: over by {float(off.max())}"


def rounded(codes, scales, x, form, name):
    """Codes stand for x within half an E4M3 step: 2^-4 of a value, 2^-10 of a scale near zero."""
    v = value(codes, scales, form)
    s = v.new_ones(()) * scales.double()
    s = s.repeat_interleave(128, -1)[..., :x.shape[-1]] if form != "col" else s
    s = s.repeat_interleave(128, -2)[..., :x.shape[-2], :] if form != "row" else s
    off = (v - x.double()).abs() - 2.0 ** -4 * x.double().abs() - 2.0 ** -10 * s * 1.001
    assert float(off.max()) <= 0, name


@pytest.mark.parametrize("T,d,f,E,R", [(300, 272, 144, 8, 2), (1024, 512, 256, 32, 4),
                                       (5, 128, 64, 16, 3)])
def test_chain_step_by_step(lib, T, d, f, E, R):
    m = load()
    gen = torch.Generator(device="cuda").manual_seed(T)
    b = m.Fp8Experts(T, d, f, E, R, gen)
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    y = b.forward(x)
    dx = b.backward(dy)
    assert torch.isfinite(y.float()).all() and torch.isfinite(dx.float()).all()
    assert (b.idx >= 0).all() and (b.idx < E).all()
    total = b.gate.sum(1)
    assert ((total - 2.0).abs() < 1e-5).all()            # renormalised, times 2
    ends = b.offsets.tolist()
    assert all(o % 128 == 0 for o in ends)
    for w in (b.w13, b.w2):
        rounded(w.q, w.s, w.w, "tile", "weights")
    for c, of, name in ((b.x_c, b.rows, "rows"), (b.h_c, b.h, "h"), (b.dout_c, b.dout, "dout"),
                        (b.dab_c, b.dab, "dab")):
        rounded(c.row, c.row_s, of, "row", name)
        rounded(c.col, c.col_s, of, "col", name)
    for e in range(E):
        i = slice(ends[e], ends[e + 1])
        blocks = slice(ends[e] // 128, ends[e + 1] // 128)
        if ends[e] == ends[e + 1]:
            assert not b.w13.grad[e].any() and not b.w2.grad[e].any()
            continue
        W13, W2 = value(b.w13.q[e], b.w13.s[e], "tile"), value(b.w2.q[e], b.w2.s[e], "tile")
        for c, W, got, t, name in ((b.x_c, W13, b.ab, True, "ab"), (b.h_c, W2, b.out, True, "out"),
                                   (b.dout_c, W2, b.dh, False, "dh"),
                                   (b.dab_c, W13, b.drows, False, "drows")):
            v = value(c.row[i], c.row_s[i], "row")
            W = W.t() if t else W
            close(got[i], v @ W, v.abs() @ W.abs(), v.shape[1], torch.bfloat16, name)
        for g, c, w, name in ((b.dab_c, b.x_c, b.w13, "dW13"), (b.dout_c, b.h_c, b.w2, "dW2")):
            gv = value(g.col[i], g.col_s[blocks], "col").t()
            cv = value(c.col[i], c.col_s[blocks], "col")
            close(w.grad[e], gv @ cv, gv.abs() @ cv.abs(), ends[e + 1] - ends[e], torch.float32, name)
    # rows behind the last expert's: never written
    for t in (b.ab, b.out, b.dh, b.drows):
        assert not t[ends[-1]:].any()


def test_gradients_against_the_block_without_rounding(lib):
    """E4M3 rounds a value by a relative error within 2^-4, evenly spread: 2^-4 / sqrt(3) in the
    mean square at most.  A gradient of the block passes through at most nine rounded operands
    (x, W13, h, W2, dout, dab, and W2, W13, x or h again on the way back): with independent
    errors 3 * 2^-4 / sqrt(3) = 0.108 of its norm; bf16 steps add below 0.01."""
    m = load()
    gen = torch.Generator(device="cuda").manual_seed(11)
    T, d, f, E, R = 512, 256, 128, 8, 2
    b = m.Fp8Experts(T, d, f, E, R, gen)
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    b.forward(x)
    dx = b.backward(dy)
    idx = b.idx.long()
    z = x.double().requires_grad_(True)
    W13, W2, wg = (t.double().requires_grad_(True) for t in (b.w13.w, b.w2.w, b.wg))
    s = torch.sigmoid(z @ wg).gather(1, idx)
    w = 2.0 * s / s.sum(1, keepdim=True)
    y = 0.0
    for r in range(R):
        a, c = torch.einsum("td,tfd->tf", z, W13[idx[:, r]]).split(f, 1)
        h = torch.nn.functional.silu(a) * c
        y = y + w[:, r, None] * torch.einsum("tf,tdf->td", h, W2[idx[:, r]])
    (y * dy.double()).sum().backward()
    for got, ref, name in ((dx, z.grad, "dx"), (b.w13.grad, W13.grad, "dW13"),
                           (b.w2.grad, W2.grad, "dW2"), (b.dwg, wg.grad, "dwg")):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err < 0.118, f"{name}: {err}"


def test_the_same_bits_again_and_from_a_graph(lib):
    m = load()
    gen = torch.Generator(device="cuda").manual_seed(3)
    b = m.Fp8Experts(256, 256, 128, 16, 2, gen)
    x = torch.randn(256, 256, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(256, 256, generator=gen, device="cuda").bfloat16()

    def step():
        y = b.forward(x)
        return (y, b.backward(dy))

    first = [t.clone() for t in step()] + [b.w13.grad.clone(), b.w2.grad.clone()]
    second = list(step()) + [b.w13.grad, b.w2.grad]
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = step()
    x.copy_(torch.randn(256, 256, generator=gen, device="cuda").bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone(), dx.clone(), b.w13.grad.clone()
    y2, dx2 = step()
    assert torch.equal(got[0], y2) and torch.equal(got[1], dx2) and torch.equal(got[2], b.w13.grad)
    assert not torch.equal(got[0], first[0])


def test_example_runs(lib, monkeypatch, capsys):
    m = load()
    monkeypatch.setattr("sys.argv", ["fp8_experts.py", "--steps", "3"])
    m.main()
    assert capsys.readouterr().out.count("step") == 3
