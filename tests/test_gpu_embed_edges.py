"""GPU: the embedding's gradient over vocabularies that take the id sort three passes."""
import pytest
import torch

from tests.test_gpu_embed import ids_of
from tests.test_gpu_sort_rows import rounded, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,V,kind", [(9001, 1_100_003, "power"), (9001, 1_100_003, "masked"),
                                      (70_000, 1_100_003, "power"), (30, 2 ** 20 + 1, "masked"),
                                      (5000, 20_000_001, "power")])
def test_three_pass_sort(lib, n, V, kind, accumulate):
    """V above 2^20, ids that repeat: against 64-bit sums; the last row among the ids."""
    d = 8
    gen = torch.Generator(device="cuda").manual_seed(n)
    ids = ids_of(n, V, kind, n, torch.int64 if n % 2 else torch.int32)
    ids[::11] = V - 1
    live = ids >= 0
    dout = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    dout[~live] = float("nan")
    before = torch.randn(V, d, generator=gen, device="cuda")
    grad = before.clone() if accumulate else torch.full_like(before, float("nan"))
    lib.moe_embed_bwd(dout, ids, grad, lib.workspace(lib.embed_bwd_ws_bytes(n, V, d)),
                      accumulate=accumulate, flags=lib.MOE_CHECK)
    at = ids[live].long()
    count = torch.bincount(at, minlength=V)[:, None].double()
    sums = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, at, dout[live].double())
    size = torch.zeros_like(sums).index_add_(0, at, dout[live].double().abs())
    if accumulate:
        sums, size = sums + before.double(), size + before.double().abs()
    within(grad, sums, rounded(sums, size, count + 3, torch.float32), "gradient")
    none = count[:, 0] == 0
    assert torch.equal(grad[none], before[none] if accumulate else torch.zeros_like(before[none]))
