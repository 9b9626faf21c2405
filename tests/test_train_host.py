"""Host-side checks of the operators around the layer: refusals, workspace
queries and the row bound answer without touching a GPU."""
import ctypes

import pytest

from expert_moe_route_gb300 import binding as B

OK, INVALID, UNSUPPORTED, WORKSPACE, BAD, _, CUDA = range(7)
P = 1 << 20     # an aligned stand-in pointer; never dereferenced


def test_rows_bound():
    bound = B.lib().moe_sort_rows_bound
    assert bound(16, 8, 64, 1, 0) == 128
    assert bound(0, 8, 64, 128, 0) == 0
    assert bound(1, 2, 8, 16, 0) == 32          # two experts with a row each, a tile each
    assert bound(100, 2, 8, 16, 0) == (200 + 8 * 15) // 16 * 16
    assert bound(100, 2, 8, 16, 10) == 8 * 16   # at most 10 rows, one tile, an expert
    assert bound(100, 2, 8, 1, 1000) == 200
    for bad in ((-1, 2, 8, 1, 0), (4, 0, 8, 1, 0), (4, 33, 64, 1, 0), (4, 2, 1025, 1, 0),
                (4, 2, 8, 0, 0), (4, 2, 8, 4097, 0), (1 << 28, 8, 8, 1, 0)):
        assert bound(*bad) == -1, bad


@pytest.mark.parametrize("T,R,E,align,cap", [(3, 2, 4, 8, 0), (7, 1, 3, 5, 2), (5, 4, 4, 3, 3),
                                             (1, 1, 1, 7, 0), (4, 3, 2, 2, 1)])
def test_rows_bound_holds_for_every_split(T, R, E, align, cap):
    """The bound is the largest sum over all ways to share the slots among the experts."""
    n = T * R

    def most(left, experts):
        if experts == 0:
            return 0
        best = 0
        for k in range(left + 1):
            kept = min(k, cap) if cap > 0 else k
            best = max(best, -(-kept // align) * align + most(left - k, experts - 1))
        return best

    got = B.sort_rows_bound(T, R, E, align, cap)
    assert got >= most(n, E)
    assert got <= most(n, E) + align * E


def test_sort_refusals():
    lib = B.lib()
    n = ctypes.c_size_t(0)

    def sort(T=8, E=8, R=2, align=1, cap=0, N=16, idx=P, counts=P, offsets=P, row_slot=P,
             slot_row=P, ws=P, nbytes=256):
        n.value = nbytes
        return lib.moe_sort(idx, T, E, R, align, cap, N, counts, offsets, row_slot, slot_row, ws,
                            ctypes.byref(n), 0, None)

    assert sort(ws=None) == OK and n.value == 256
    assert sort(T=-1) == INVALID and sort(R=0) == INVALID and sort(E=0) == INVALID
    assert sort(align=0) == INVALID and sort(align=5000) == UNSUPPORTED
    assert sort(R=33) == UNSUPPORTED and sort(E=1025) == UNSUPPORTED
    assert sort(N=15) == INVALID                       # fewer rows than the plan may need
    assert sort(nbytes=255) == WORKSPACE and sort(ws=P + 16) == WORKSPACE
    for name in ("idx", "counts", "offsets", "row_slot", "slot_row"):
        assert sort(**{name: None}) == INVALID, name
        assert sort(**{name: P + 2}) == UNSUPPORTED, name
    assert lib.moe_sort(P, 8, 8, 2, 1, 0, 16, P, P, P, P, P, None, 0, None) == INVALID


def test_row_mover_refusals():
    lib = B.lib()

    def permute(x=P, ldx=64, w=P, row_slot=P, slot_row=P, T=8, d=64, R=2, N=16, dtype=0, rows=P,
                ldr=64):
        return lib.moe_permute(x, ldx, w, row_slot, slot_row, T, d, R, N, dtype, rows, ldr, None)

    def back(dy=P, ldy=64, row_slot=P, slot_row=P, w=P, rows=P, ldr=64, T=8, d=64, R=2, N=16,
             dtype=0, drows=P, ldd=64, dw=P):
        return lib.moe_unpermute_bwd(dy, ldy, row_slot, slot_row, w, rows, ldr, T, d, R, N, dtype,
                                     drows, ldd, dw, None)

    def grad(drows=P, ldr=64, slot_row=P, w=P, x=P, ldx=64, T=8, d=64, R=2, N=16, dtype=0, dx=P,
             ldd=64, dw=P):
        return lib.moe_permute_bwd(drows, ldr, slot_row, w, x, ldx, T, d, R, N, dtype, dx, ldd, dw,
                                   None)

    def unpermute(rows=P, ldr=64, slot_row=P, w=P, T=8, d=64, R=2, N=16, dtype=0, y=P, ldy=64):
        return lib.moe_unpermute(rows, ldr, slot_row, w, T, d, R, N, dtype, y, ldy, None)

    for f in (permute, back, grad, unpermute):
        assert f(T=-1) == INVALID and f(d=0) == INVALID and f(R=0) == INVALID and f(N=-1) == INVALID
        assert f(dtype=3) == INVALID
        assert f(R=33) == UNSUPPORTED
        assert f(slot_row=None) == INVALID and f(slot_row=P + 1) == UNSUPPORTED
        assert f(w=P + 2) == UNSUPPORTED
    assert permute(x=None) == INVALID and permute(rows=None) == INVALID
    assert permute(row_slot=None) == INVALID
    assert permute(ldx=63) == INVALID and permute(ldr=63) == INVALID
    assert permute(x=P + 1) == UNSUPPORTED and permute(rows=P + 2, dtype=2) == UNSUPPORTED
    assert back(dw=None) == INVALID and back(rows=None) == INVALID     # both or neither
    assert grad(dw=None) == INVALID and grad(x=None) == INVALID
    assert grad(ldx=1) == INVALID and grad(dw=P + 2) == UNSUPPORTED
    assert unpermute(y=None) == INVALID and unpermute(ldy=8) == INVALID


def test_embedding_refusals():
    lib = B.lib()
    n = ctypes.c_size_t(0)

    def embed(ids=P, ib=8, n_=16, table=P, ldt=64, V=100, d=64, tt=0, out=P, ldo=64, ot=0):
        return lib.moe_embed(ids, ib, n_, table, ldt, V, d, tt, 1.0, out, ldo, ot, None)

    def grad(dout=P, ldd=64, ids=P, ib=8, n_=16, V=100, d=64, dt=0, dtable=P, ldt=64, tt=2, ws=P,
             nbytes=1 << 30):
        n.value = nbytes
        return lib.moe_embed_bwd(dout, ldd, ids, ib, n_, V, d, dt, 1.0, dtable, ldt, tt, ws,
                                 ctypes.byref(n), 0, None)

    for f in (embed, grad):
        assert f(n_=-1) == INVALID and f(V=0) == INVALID and f(d=0) == INVALID
        assert f(ib=2) == INVALID and f(tt=7) == INVALID
        assert f(ids=None) == INVALID and f(ids=P + 4) == UNSUPPORTED
        assert f(ldt=63) == INVALID
    assert embed(n_=0) == OK
    assert embed(table=None) == INVALID and embed(out=None) == INVALID
    assert embed(n_=1 << 31) == UNSUPPORTED
    assert grad(ws=None) == OK and n.value > 256
    assert grad(nbytes=256) == WORKSPACE and grad(ws=P + 16) == WORKSPACE
    assert grad(dout=None) == INVALID and grad(dtable=None) == INVALID
    assert grad(n_=1 << 30) == UNSUPPORTED


def test_optimiser_refusals():
    lib = B.lib()
    good = dict(p=P, master=None, g=P, m=P, v=P, m_scale=None, v_scale=None, n=100,
                weight_decay=0.1, p_dtype=0, g_dtype=2, state_bits=32)
    settings = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0)
    n = ctypes.c_size_t(0)

    def step(norm=None, hyper=None, **changes):
        x = (B.moe_adamw_tensor_t * 1)(B.moe_adamw_tensor_t(**{**good, **changes}))
        h = B.moe_adamw_t(**{**settings, **(hyper or {})})
        return lib.moe_adamw_step(x, 1, ctypes.byref(h), norm, None)

    def norm(out=P, ws=P, nbytes=1 << 20, max_norm=1.0, **changes):
        x = (B.moe_adamw_tensor_t * 1)(B.moe_adamw_tensor_t(**{**good, **changes}))
        n.value = nbytes
        return lib.moe_grad_norm(x, 1, max_norm, out, ws, ctypes.byref(n), None)

    for f in (step, norm):
        assert f(n=-1) == INVALID and f(g=None) == INVALID
        assert f(g=P + 2) == UNSUPPORTED and f(g_dtype=1) == UNSUPPORTED
        assert f(n=1 << 40) == UNSUPPORTED
    for name in ("p", "m", "v"):
        assert step(**{name: None}) == INVALID
    assert step(p=P + 1) == UNSUPPORTED and step(m=P + 2) == UNSUPPORTED
    assert step(p_dtype=1) == UNSUPPORTED and step(state_bits=16) == UNSUPPORTED
    assert step(state_bits=8) == INVALID                              # no scales
    assert step(master=P, p_dtype=2) == INVALID                       # an fp32 p is its own master
    assert step(weight_decay=float("nan")) == INVALID
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(step=0),
                dict(lr=float("inf")), dict(beta1=float("nan")), dict(eps=1e-60)):
        assert step(hyper=bad) == INVALID, bad
    assert step(norm=P + 4) == UNSUPPORTED
    assert lib.moe_adamw_step(None, 1, None, None, None) == INVALID
    assert lib.moe_adamw_step(None, 0, None, None, None) == INVALID   # no settings
    assert norm(ws=None) == OK and n.value > 0
    assert norm(nbytes=8) == WORKSPACE and norm(ws=P + 8) == WORKSPACE
    assert norm(out=None) == INVALID and norm(max_norm=float("nan")) == INVALID


def test_binding_refuses_wrong_types():
    torch = pytest.importorskip("torch")
    p, g = torch.zeros(512), torch.zeros(512)
    m = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(TypeError):
        B.AdamWTensor(p, g.half(), p, p)
    with pytest.raises(TypeError):
        B.AdamWTensor(p, g, p, m)
    with pytest.raises(ValueError):
        B.AdamWTensor(p, g, m, m)                       # 8-bit states need scales
    with pytest.raises(ValueError):
        B.AdamWTensor(p, g[:100], p, p)
    with pytest.raises(ValueError):
        B.AdamWTensor(p, g, m, m, m_scale=torch.zeros(1), v_scale=torch.zeros(2))
    with pytest.raises(TypeError):
        B.moe_embed(torch.zeros(4), p.view(8, 64), p.view(8, 64))
