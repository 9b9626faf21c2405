"""One training step around the MoE layer, with the library's operators only where
the work is and torch for the rest: token ids -> embedding -> the MoE layer -> a
second block whose experts are this file's own (squared ReLU) -> loss -> gradients
-> gradient norm -> AdamW on every parameter.

    python examples/train_step.py [--steps 30] [--states 8]

Learns to map each token to a fixed random vector; prints the loss of each step.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from expert_moe_route_gb300 import binding as B  # noqa: E402

BF, F = torch.bfloat16, torch.float32


class OwnExperts:
    """y = x + sum_r w_r expert_r(x), expert_e(row) = relu(row A_e)^2 B_e: rows sorted by expert with
    moe_sort / moe_permute, brought back with moe_unpermute; a fixed number of rows an expert."""

    def __init__(self, T, d, f, E, R, gen):
        self.T, self.d, self.E, self.R = T, d, E, R
        dev = dict(device="cuda")
        self.wg = torch.randn(d, E, generator=gen, **dev) * 0.02
        self.A = (torch.randn(E, d, f, generator=gen, **dev) / math.sqrt(d)).to(BF)
        self.B = (torch.randn(E, f, d, generator=gen, **dev) / math.sqrt(f)).to(BF)
        # every expert takes at most `align` rows: with capacity == align its segment, when it has
        # any row, is exactly one tile
        self.align = self.capacity = -(-2 * T * R // E // 16) * 16
        self.N = B.sort_rows_bound(T, R, E, self.align, self.capacity)
        i32 = dict(dtype=torch.int32, **dev)
        self.logits = torch.empty(T, E, **dev)
        self.idx, self.w = torch.empty(T, R, **i32), torch.empty(T, R, **dev)
        self.counts, self.offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        self.row_slot, self.slot_row = torch.empty(self.N, **i32), torch.empty(T, R, **i32)
        self.route_ws = B.workspace(B.route_ws_bytes(T, d, E, R))
        self.sort_ws = B.workspace(B.sort_ws_bytes(T, E, R))
        self.rows = torch.empty(self.N, d, dtype=BF, **dev)
        self.out = torch.zeros(self.N, d, dtype=BF, **dev)
        self.dA, self.dB = torch.zeros_like(self.A, dtype=F), torch.zeros_like(self.B, dtype=F)
        self.dwg = torch.zeros_like(self.wg)

    def forward(self, x):
        B.moe_route(x, self.wg, None, self.logits, self.idx, self.w, self.route_ws)
        B.moe_sort(self.idx, self.E, self.counts, self.offsets, self.row_slot, self.slot_row,
                   self.sort_ws, align=self.align, capacity=self.capacity)
        B.moe_permute(x, None, self.row_slot, self.slot_row, self.rows)
        # one tile an expert that has rows: the tiles' experts, in row order
        self.tile_expert = torch.nonzero(self.counts)[:, 0]
        tiles = self.rows[:self.tile_expert.numel() * self.align].view(-1, self.align, self.d)
        self.pre = torch.bmm(tiles, self.A[self.tile_expert])
        self.hidden = torch.relu(self.pre) ** 2
        self.out[:tiles.shape[0] * self.align] = torch.bmm(
            self.hidden, self.B[self.tile_expert]).view(-1, self.d)
        y = torch.empty_like(x)
        B.moe_unpermute(self.out, self.slot_row, self.w, y)
        self.x = x
        return x + y

    def backward(self, dy):
        drows, dw = torch.empty_like(self.rows), torch.empty_like(self.w)
        B.moe_unpermute_bwd(dy, self.row_slot, self.slot_row, self.w, self.out, drows, dw)
        n = self.tile_expert.numel() * self.align
        dout = drows[:n].view(-1, self.align, self.d)
        tiles = self.rows[:n].view(-1, self.align, self.d)
        At, Bt = self.A[self.tile_expert], self.B[self.tile_expert]
        dpre = torch.bmm(dout, Bt.transpose(1, 2)) * 2 * torch.relu(self.pre)
        self.dA.zero_()
        self.dB.zero_()
        self.dA[self.tile_expert] = torch.bmm(tiles.transpose(1, 2), dpre).float()
        self.dB[self.tile_expert] = torch.bmm(self.hidden.transpose(1, 2), dout).float()
        drows[:n] = torch.bmm(dpre, At.transpose(1, 2)).view(-1, self.d)
        dx = torch.empty_like(dy)
        B.moe_permute_bwd(drows, self.slot_row, None, None, dx, None)
        # the gate weights are a softmax over the chosen logits
        dl = torch.zeros(self.T, self.E, device="cuda")
        dl.scatter_(1, self.idx.long(), self.w * (dw - (self.w * dw).sum(1, keepdim=True)))
        torch.mm(self.x.float().t(), dl, out=self.dwg)
        return (dy.float() + dx.float() + dl @ self.wg.t()).to(BF)

    def parameters(self):
        return [(self.wg, self.dwg), (self.A, self.dA), (self.B, self.dB)]


class Layer:
    """y = x + the library's MoE layer (SwiGLU experts)."""

    def __init__(self, T, d, f, E, R, gen):
        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") / math.sqrt(shape[-1])).to(BF)

        self.wg = torch.randn(d, E, generator=gen, device="cuda") * 0.02
        self.W1, self.W3, self.W2 = weight(E, f, d), weight(E, f, d), weight(E, d, f)
        self.layer = B.Layer(self.wg, None, self.W1, self.W3, self.W2, R, T)
        self.saved = B.Saved(self.layer, "cuda", train=True)
        self.fwd_ws = B.workspace(B.layer_fwd_ws_bytes(self.layer))
        self.bwd_ws = B.workspace(B.layer_bwd_ws_bytes(self.layer))
        self.grads = [torch.empty_like(t, dtype=F) for t in (self.wg, self.W1, self.W3, self.W2)]

    def forward(self, x):
        self.x = x
        y = torch.empty_like(x)
        B.moe_layer_fwd(self.layer, x, y, self.saved, self.fwd_ws)
        return x + y

    def backward(self, dy):
        dx = torch.empty_like(dy)
        B.moe_layer_bwd(self.layer, self.x, self.saved, dy, dx, *self.grads, self.bwd_ws)
        return dy + dx

    def parameters(self):
        return list(zip((self.wg, self.W1, self.W3, self.W2), self.grads))


class Training:
    def __init__(self, V=1000, T=512, d=256, f=256, E=16, R=2, states=8, lr=3e-3, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.V, self.T, self.d = gen, V, T, d
        self.table = torch.randn(V, d, generator=gen, device="cuda") * 0.02
        self.dtable = torch.empty_like(self.table)
        self.scale = math.sqrt(d)
        self.embed_ws = B.workspace(B.embed_bwd_ws_bytes(T, V, d))
        self.goal = torch.randn(V, d, generator=gen, device="cuda")
        self.blocks = [Layer(T, d, f, E, R, gen), OwnExperts(T, d, f, E, R, gen)]
        pairs = [(self.table, self.dtable)]
        for b in self.blocks:
            pairs += b.parameters()
        self.list = B.AdamWList([self.state(p, g, states) for p, g in pairs])
        self.norm = torch.empty(4, device="cuda")
        self.norm_ws = B.workspace(B.grad_norm_ws_bytes(self.list))
        self.lr, self.step_number = lr, 0

    @staticmethod
    def state(p, g, states):
        n = p.numel()
        dev = dict(device="cuda")
        master = p.float() if p.dtype == BF else None
        decay = 0.01 if p.dim() > 1 else 0.0
        if states == 32:
            return B.AdamWTensor(p, g, torch.zeros(n, **dev), torch.zeros(n, **dev), master=master,
                                 weight_decay=decay)
        m, v = (torch.zeros(n, dtype=torch.uint8, **dev) for _ in range(2))
        ms, vs = (torch.zeros(-(-n // 256), **dev) for _ in range(2))
        return B.AdamWTensor(p, g, m, v, master=master, m_scale=ms, v_scale=vs, weight_decay=decay)

    def step(self):
        """One step on new tokens; returns the loss (a device scalar)."""
        u = torch.rand(self.T, generator=self.gen, device="cuda")
        ids = (torch.exp(u * math.log(self.V + 1)).long() - 1).clamp_(0, self.V - 1)
        x = torch.empty(self.T, self.d, dtype=BF, device="cuda")
        B.moe_embed(ids, self.table, x, scale=self.scale)
        for b in self.blocks:
            x = b.forward(x)
        diff = x.float() - self.goal[ids]
        loss = 0.5 * diff.square().mean()
        dy = (diff / diff.numel()).to(BF)
        for b in reversed(self.blocks):
            dy = b.backward(dy)
        B.moe_embed_bwd(dy, ids, self.dtable, self.embed_ws, scale=self.scale)
        self.step_number += 1
        B.moe_grad_norm(self.list, 1.0, self.norm, self.norm_ws)
        B.moe_adamw_step(self.list, self.lr, beta2=0.98, step=self.step_number,
                         seed=self.step_number, norm=self.norm)
        return loss


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--states", type=int, choices=(8, 32), default=8)
    args = ap.parse_args()
    run = Training(states=args.states)
    for k in range(args.steps):
        print(f"step {k + 1:3d}  loss {float(run.step()):.4f}  gradient norm {float(run.norm[0]):.3f}")


if __name__ == "__main__":
    main()
