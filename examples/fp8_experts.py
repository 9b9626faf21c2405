"""An MoE block whose experts compute in block-scaled fp8, forward and backward, with its
router: sigmoid scores, a balance bias, groups -> rows sorted by expert -> E4M3 codes ->
the experts' products on the fp8 tensor cores -> rows back, and the gradients of all of it.
torch does what is left: the gate's product, SwiGLU, the loss.

    python examples/fp8_experts.py [--steps 20]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from expert_moe_route_gb300 import binding as B  # noqa: E402

BF, F, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


class Codes:
    """A matrix's codes by row (for products) and by column (for weights' gradients)."""

    def __init__(self, N, K):
        self.row, self.col = (torch.empty(N, K, dtype=E4M3, device="cuda") for _ in "rc")
        self.row_s = torch.empty(N, B.fp8_blocks(K), device="cuda")
        self.col_s = torch.empty(B.fp8_blocks(N), K, device="cuda")

    def of(self, x):
        B.moe_quantize_fp8(x, self.row, self.row_s, self.col, self.col_s)
        return self


class Weights:
    """bf16 weights [E, n, K] with their codes, made anew each step, and their gradient."""

    def __init__(self, E, n, K, gen):
        self.w = (torch.randn(E, n, K, generator=gen, device="cuda") / math.sqrt(K)).to(BF)
        self.q = torch.empty(E, n, K, dtype=E4M3, device="cuda")
        self.s = torch.empty(E, B.fp8_blocks(n), B.fp8_blocks(K), device="cuda")
        self.grad = torch.empty(E, n, K, device="cuda")

    def quantize(self):
        B.moe_quantize_fp8_tiles(self.w, self.q, self.s)


class Fp8Experts:
    """y = sum_r w_r expert_r(x), expert(row) = (silu(row A^T) * (row C^T)) W2^T with W13 = [A; C]."""

    def __init__(self, T, d, f, E, R, gen, router=None):
        self.T, self.d, self.f, self.E, self.R = T, d, f, E, R
        self.router = router or B.Router(score="sigmoid", groups=4, top_groups=2, group_keys=2,
                                         scale=2.0)
        self.wg = torch.randn(d, E, generator=gen, device="cuda") / math.sqrt(d)
        self.dwg = torch.empty_like(self.wg)
        self.bias = torch.zeros(E, device="cuda")
        self.w13, self.w2 = Weights(E, 2 * f, d, gen), Weights(E, d, f, gen)
        self.N = N = B.sort_rows_bound(T, R, E, align=128)    # blocks of 128 rows have one expert
        i32 = dict(dtype=I32, device="cuda")
        self.idx, self.counts = torch.empty(T, R, **i32), torch.empty(E, **i32)
        self.offsets, self.row_slot = torch.empty(E + 1, **i32), torch.empty(N, **i32)
        self.slot_row = torch.empty(T, R, **i32)
        self.gate, self.dgate = torch.empty(T, R, device="cuda"), torch.empty(T, R, device="cuda")
        self.dlogits = torch.empty(T, E, device="cuda")
        self.sort_ws = B.workspace(B.sort_ws_bytes(T, E, R))
        self.ws = B.workspace(max(B.product_fp8_ws_bytes(N, 2 * f, d, E),
                                  B.product_fp8_ws_bytes(N, d, f, E)))

        def rows(width):       # rows behind the last expert's are never written: zeros
            return torch.zeros(N, width, dtype=BF, device="cuda")

        self.rows, self.ab, self.out = rows(d), rows(2 * f), rows(d)
        self.dout, self.dh, self.drows = rows(d), rows(f), rows(d)
        self.x_c, self.h_c, self.dout_c, self.dab_c = (Codes(N, k) for k in (d, f, d, 2 * f))

    def forward(self, x):
        self.w13.quantize()
        self.w2.quantize()
        self.x = x
        self.logits = x.float() @ self.wg
        B.moe_route_scores(self.logits, self.router, self.idx, self.gate, bias=self.bias)
        B.moe_sort(self.idx, self.E, self.counts, self.offsets, self.row_slot, self.slot_row,
                   self.sort_ws, align=128)
        B.moe_permute(x, None, self.row_slot, self.slot_row, self.rows)
        c = self.x_c.of(self.rows)
        B.moe_product_fp8(c.row, c.row_s, self.w13.q, self.w13.s, self.ab, self.ws, self.offsets)
        a, b = self.ab.float().split(self.f, 1)
        self.h = (torch.nn.functional.silu(a) * b).to(BF)
        c = self.h_c.of(self.h)
        B.moe_product_fp8(c.row, c.row_s, self.w2.q, self.w2.s, self.out, self.ws, self.offsets)
        y = torch.empty_like(x)
        B.moe_unpermute(self.out, self.slot_row, self.gate, y)
        return y

    def backward(self, dy):
        B.moe_unpermute_bwd(dy, self.row_slot, self.slot_row, self.gate, self.out, self.dout,
                            self.dgate)
        c = self.dout_c.of(self.dout)
        B.moe_product_fp8_dx(c.row, c.row_s, self.w2.q, self.w2.s, self.dh, self.ws, self.offsets)
        B.moe_product_fp8_dw(c.col, c.col_s, self.h_c.col, self.h_c.col_s, self.w2.grad, self.ws,
                             self.offsets)
        a, b = self.ab.float().split(self.f, 1)
        s, dh = torch.sigmoid(a), self.dh.float()
        self.dab = torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], 1).to(BF)
        c = self.dab_c.of(self.dab)
        B.moe_product_fp8_dx(c.row, c.row_s, self.w13.q, self.w13.s, self.drows, self.ws,
                             self.offsets)
        B.moe_product_fp8_dw(c.col, c.col_s, self.x_c.col, self.x_c.col_s, self.w13.grad, self.ws,
                             self.offsets)
        dx = torch.empty_like(dy)
        B.moe_permute_bwd(self.drows, self.slot_row, None, None, dx, None)
        B.moe_route_scores_bwd(self.logits, self.router, self.idx, self.dgate, self.dlogits)
        torch.mm(self.x.float().t(), self.dlogits, out=self.dwg)
        return (dx.float() + self.dlogits @ self.wg.t()).to(BF)

    def balance(self, rate=1e-3):
        """Experts with more rows than the mean lose a little of their bias, the others gain it."""
        load = self.counts.float()
        self.bias += rate * torch.sign(load.mean() - load)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    block = Fp8Experts(2048, 512, 256, 32, 4, gen)
    goal = torch.randn(2048, 512, generator=gen, device="cuda")
    x = torch.randn(2048, 512, generator=gen, device="cuda").to(BF)
    for k in range(args.steps):
        diff = block.forward(x).float() - goal
        block.backward((diff / 64).to(BF))
        for w in (block.w13, block.w2):
            w.w -= (0.5 * w.grad).to(BF)
        block.wg -= 0.5 * block.dwg
        block.balance()
        print(f"step {k + 1:3d}  loss {0.5 * float(diff.square().mean()):.4f}  "
              f"largest expert {int(block.counts.max())} rows")


if __name__ == "__main__":
    main()
