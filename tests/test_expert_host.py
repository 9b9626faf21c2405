"""Host-side checks of routing by scores and of the products on block-scaled fp8: refusals and
workspace queries answer without touching a GPU."""
import ctypes

import pytest
import torch

from expert_moe_route_gb300 import binding as B

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
P = 1 << 20     # an aligned stand-in pointer; never dereferenced


def router(score=1, groups=4, top_groups=2, group_keys=2, renormalise=1, scale=2.5):
    return ctypes.byref(B.moe_router_t(score, groups, top_groups, group_keys, renormalise, scale))


def test_route_scores_refusals():
    lib = B.lib()

    def fwd(logits=P, ld=64, dtype=2, bias=P, T=8, E=64, R=4, r=None, idx=P, w=P):
        return lib.moe_route_scores(logits, ld, dtype, bias, T, E, R, r or router(), idx, w, None)

    def bwd(logits=P, ld=64, dtype=2, idx=P, dw=P, T=8, E=64, R=4, r=None, out=P, ldo=64):
        return lib.moe_route_scores_bwd(logits, ld, dtype, idx, dw, T, E, R, r or router(), out,
                                        ldo, None)

    for f in (fwd, bwd):
        assert f(T=-1) == INVALID and f(E=0) == INVALID and f(R=0) == INVALID
        assert f(dtype=3) == INVALID and f(logits=None) == INVALID and f(ld=63) == INVALID
        assert f(idx=None) == INVALID and f(idx=P + 2) == UNSUPPORTED
        assert f(logits=P + 2) == UNSUPPORTED
        assert f(R=33, E=64, r=router(groups=1, top_groups=1, group_keys=1)) == UNSUPPORTED
        assert f(E=1028, ld=1028) == UNSUPPORTED
        assert f(T=1 << 30, R=2) == UNSUPPORTED
        assert f(R=33, E=1024, ld=1024) == UNSUPPORTED
        assert f(r=router(score=2)) == INVALID
        assert f(r=router(groups=0)) == INVALID and f(r=router(groups=5)) == INVALID
        assert f(r=router(groups=64, top_groups=64, group_keys=1)) == UNSUPPORTED
        assert f(r=router(top_groups=0)) == INVALID and f(r=router(top_groups=5)) == INVALID
        assert f(r=router(group_keys=0)) == INVALID and f(r=router(group_keys=3)) == INVALID
        assert f(r=router(groups=32, top_groups=32, group_keys=2), E=32, ld=32) == INVALID
        assert f(R=17, r=router(top_groups=1)) == INVALID       # 16 experts in one group
        assert f(r=router(scale=float("nan"))) == INVALID
        assert f(r=router(scale=float("inf"))) == INVALID
    assert fwd(w=None) == INVALID and fwd(w=P + 1) == UNSUPPORTED and fwd(bias=P + 2) == UNSUPPORTED
    assert bwd(dw=None) == INVALID and bwd(out=None) == INVALID and bwd(ldo=63) == INVALID
    assert lib.moe_route_scores(P, 64, 2, None, 8, 64, 4, None, P, P, None) == INVALID
    assert fwd(T=0, logits=None, idx=None, w=None) == OK
    assert bwd(T=0, logits=None, idx=None, dw=None, out=None) == OK


def test_quantize_refusals():
    lib = B.lib()

    def rows(x=P, ldx=64, dtype=0, N=8, K=64, rc=P, rs=P, cc=P, cs=P):
        return lib.moe_quantize_fp8(x, ldx, dtype, N, K, rc, rs, cc, cs, None)

    def tiles(w=P, dtype=0, E=2, n=64, K=64, codes=P, scales=P):
        return lib.moe_quantize_fp8_tiles(w, dtype, E, n, K, codes, scales, None)

    assert rows(N=-1) == INVALID and rows(K=0) == INVALID and rows(dtype=9) == INVALID
    assert rows(x=None) == INVALID and rows(ldx=63) == INVALID and rows(x=P + 1) == UNSUPPORTED
    assert rows(K=24, ldx=24) == UNSUPPORTED and rows(N=(1 << 30) + 1) == UNSUPPORTED
    assert rows(rc=None) == INVALID and rows(rs=None) == INVALID     # codes go with scales
    assert rows(cc=None) == INVALID and rows(cs=None) == INVALID
    assert rows(rc=None, rs=None, cc=None, cs=None) == INVALID
    assert rows(rc=P + 8) == UNSUPPORTED and rows(cc=P + 4) == UNSUPPORTED
    assert rows(rs=P + 2) == UNSUPPORTED and rows(cs=P + 1) == UNSUPPORTED
    assert rows(N=0, x=None, rc=None, rs=None, cc=None, cs=None) == OK
    assert tiles(E=-1) == INVALID and tiles(n=0) == INVALID and tiles(K=0) == INVALID
    assert tiles(dtype=4) == INVALID and tiles(K=40) == UNSUPPORTED
    assert tiles(w=None) == INVALID and tiles(codes=None) == INVALID and tiles(scales=None) == INVALID
    assert tiles(w=P + 1) == UNSUPPORTED and tiles(codes=P + 8) == UNSUPPORTED
    assert tiles(scales=P + 2) == UNSUPPORTED
    assert tiles(E=0, w=None, codes=None, scales=None) == OK


def test_product_refusals():
    lib = B.lib()
    n_ = ctypes.c_size_t(0)

    def call(f, a=P, sa=P, off=P, N=256, n=64, K=128, E=2, b=P, sb=P, out=P, ld=None, dtype=0,
             ws=P, nbytes=1 << 30, back=False):
        n_.value = nbytes
        ld = (K if back else n) if ld is None else ld
        return f(a, sa, off, N, n, K, E, b, sb, out, ld, dtype, ws, ctypes.byref(n_), 0, None)

    def fwd(**k):
        return call(lib.moe_product_fp8, **k)

    def dx(**k):
        return call(lib.moe_product_fp8_dx, back=True, **k)

    def dw(a=P, sa=P, b=P, sb=P, off=P, N=256, n=64, K=128, E=2, out=P, dtype=2, ws=P,
           nbytes=1 << 30):
        n_.value = nbytes
        return lib.moe_product_fp8_dw(a, sa, b, sb, off, N, n, K, E, out, dtype, ws,
                                      ctypes.byref(n_), 0, None)

    for f in (fwd, dx, dw):
        assert f(ws=None) == OK and n_.value >= 256
        assert f(nbytes=255) == WORKSPACE and f(ws=P + 16) == WORKSPACE
        assert f(N=-1) == INVALID and f(n=0) == INVALID and f(K=0) == INVALID and f(E=0) == INVALID
        assert f(n=24) == UNSUPPORTED and f(K=136) == UNSUPPORTED and f(E=1025) == UNSUPPORTED
        assert f(N=(1 << 30) + 1) == UNSUPPORTED
        assert f(off=None) == INVALID                     # two experts need offsets
        assert f(off=P + 2) == UNSUPPORTED
        assert f(a=None) == INVALID and f(sa=None) == INVALID
        assert f(b=None) == INVALID and f(sb=None) == INVALID and f(out=None) == INVALID
        assert f(a=P + 8) == UNSUPPORTED and f(b=P + 8) == UNSUPPORTED
        assert f(sa=P + 2) == UNSUPPORTED and f(sb=P + 2) == UNSUPPORTED
        assert f(dtype=3) == INVALID
    assert fwd(ld=63) == INVALID and dx(ld=127) == INVALID
    assert fwd(out=P + 1) == UNSUPPORTED and dw(out=P + 8) == UNSUPPORTED
    assert dw(sb=P + 4) == UNSUPPORTED
    assert fwd(N=0, a=None, sa=None, out=None) == OK      # nothing to do


@pytest.mark.parametrize("N,n,K,E", [(1, 2048, 4096, 1), (128, 256, 512, 4), (64, 64, 8192, 1),
                                     (4096, 256, 256, 1)])
def test_workspace_is_one_size_for_the_three(N, n, K, E):
    lib = B.lib()
    got = []
    for f in (lib.moe_product_fp8, lib.moe_product_fp8_dx):
        s = ctypes.c_size_t(0)
        assert f(None, None, None, N, n, K, E, None, None, None, n, 0, None, ctypes.byref(s), 0,
                 None) == OK
        got.append(s.value)
    s = ctypes.c_size_t(0)
    assert lib.moe_product_fp8_dw(None, None, None, None, None, N, n, K, E, None, 2, None,
                                  ctypes.byref(s), 0, None) == OK
    got.append(s.value)
    assert len(set(got)) == 1
    assert got[0] <= 256 + 3 * (152 * 128 * 256 * 4)      # split tiles: at most one an SM


def test_router_names():
    with pytest.raises(ValueError):
        B.Router(score="linear")
    r = B.Router(score="sigmoid", groups=8, top_groups=4, group_keys=2, scale=2.5)
    assert (r.c.score, r.c.groups, r.c.top_groups, r.c.group_keys, r.c.renormalise, r.c.scale) == (
        1, 8, 4, 2, 1, 2.5)


def test_binding_needs_device_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        B.moe_route_scores(x, B.Router(), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        B.moe_quantize_fp8(x, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1))
    with pytest.raises(ValueError):
        B.moe_quantize_fp8_tiles(torch.zeros(1, 4, 64), torch.zeros(1, 4, 64, dtype=torch.uint8),
                                 torch.zeros(1, 1, 1))
