"""A small predictor in front of the splatting layer, trained end to end.

Features of a grid of cells pass through a projection, gated feed-forward
blocks and a head to the raw values of one Gaussian per cell, which are
activated, rendered and compared with target frames; the matrices are trained
by Muon, everything else by AdamW.  Every product, the rendering, the loss and
the optimiser's Newton-Schulz steps run in this package's kernels.  With
--heads the blocks are those of a transformer: in each, the cells of a frame
attend to one another, before the feed-forward part.

    python examples/fit_predictor.py --steps 60
    python examples/fit_predictor.py --steps 60 --heads 4 --kv-heads 2 --dropout 0.1
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_gaussian_splatting_pdr_amd import blocks as ops, dense, splat  # noqa: E402


class Predictor(torch.nn.Module):
    """features [B, gx * gy, F] -> frames [B, H, W, C]."""

    def __init__(self, features, width, hidden, blocks, gx, gy, H, W, C, dtype=torch.bfloat16,
                 device="cuda", heads=0, kv_heads=None, p=0.0):
        super().__init__()
        self.heads, self.p = heads, p
        self.grid, self.frame, self.C, self.dtype = (gx, gy), (H, W), C, dtype

        def weight(rows, cols, scale=1.0):
            return torch.nn.Parameter(torch.randn(rows, cols, device=device) * scale * cols ** -0.5)

        self.w_embed = weight(width, features)
        self.b_embed = torch.nn.Parameter(torch.zeros(width, device=device))
        self.w_in = torch.nn.ParameterList(weight(2 * hidden, width) for _ in range(blocks))
        self.w_out = torch.nn.ParameterList(weight(width, hidden, 0.5) for _ in range(blocks))
        self.w_head = weight(5 + C, width, 0.1)
        self.b_head = torch.nn.Parameter(torch.zeros(5 + C, device=device))
        if heads:
            self.kv_heads, self.head = kv_heads or heads, width // heads
            of_keys = self.kv_heads * self.head
            self.w_qkv = torch.nn.ParameterList(weight(heads * self.head + 2 * of_keys, width) for _ in range(blocks))
            self.w_mix = torch.nn.ParameterList(weight(width, heads * self.head, 0.5) for _ in range(blocks))
            self.norms = torch.nn.ParameterList(torch.nn.Parameter(t) for _ in range(2 * blocks)
                                                for t in (torch.ones(width, device=device),
                                                          torch.zeros(width, device=device)))

    def matrices(self):
        return [p for p in self.parameters() if p.dim() == 2]

    def norm(self, x, which):
        weight, bias = self.norms[2 * which], self.norms[2 * which + 1]
        return ops.layer_norm(x, weight.to(x.dtype), bias.to(x.dtype))

    def mixed(self, x, block, seed):
        """x + what each cell takes from the others of its frame."""
        d, h, hk = x.dtype, self.heads, self.kv_heads
        qkv = dense.linear(self.norm(x, 2 * block), self.w_qkv[block].to(d))
        q, k, v = qkv.view(*x.shape[:-1], h + 2 * hk, self.head).split((h, hk, hk), dim=-2)
        y = ops.attention(q, k, v)
        w = self.w_mix[block].to(d)
        if seed is None or not self.p:
            return dense.linear(y.flatten(-2), w, residual=x)
        return ops.dropout(dense.linear(y.flatten(-2), w), self.p, seed, offset=block, residual=x)

    def raw(self, x, seed=None):
        """seed: of the dropped values; None: none are."""
        d = self.dtype
        x = dense.linear(x.to(d), self.w_embed.to(d), self.b_embed.to(d), activation="gelu")
        for block, (w_in, w_out) in enumerate(zip(self.w_in, self.w_out)):
            if self.heads:
                x = self.mixed(x, block, seed)
            y = self.norm(x, 2 * block + 1) if self.heads else x
            x = dense.gated_mlp(y, w_in.to(d), w_out.to(d), residual=x)
        # the head keeps its sums' 32 bits for the renderer, on top of the grid's own Gaussians
        gx, gy = self.grid
        start = splat.grid_init(x.shape[0], gx, gy, *self.frame, self.C, device=x.device)
        return dense.linear(x, self.w_head.to(d), self.b_head.to(d), residual=start,
                            out_dtype=torch.float32)

    def forward(self, x, seed=None):
        gx, gy = self.grid
        params = splat.activate(self.raw(x, seed), gx, gy, *self.frame)
        return splat.render(params, *self.frame)


def train(steps=60, B=8, gx=16, gy=16, H=64, W=64, C=3, features=48, width=256, hidden=704,
          blocks=2, seed=0, report=None, heads=0, kv_heads=None, dropout=0.0):
    """Fit frames of a teacher of the same shape; returns the losses."""
    torch.manual_seed(seed)
    net = Predictor(features, width, hidden, blocks, gx, gy, H, W, C, heads=heads, kv_heads=kv_heads, p=dropout)
    x = torch.randn(B, gx * gy, features, device="cuda")
    with torch.no_grad():
        # smooth target frames: each cell's Gaussian carries an amplitude of its own
        start = splat.grid_init(B, gx, gy, H, W, C)
        start[..., 5:] = torch.tanh(x[..., :C])
        target = splat.render(splat.activate(start, gx, gy, H, W), H, W)
    muon = dense.Muon(net.matrices(), lr=0.02, work_dtype=torch.bfloat16)
    adam = torch.optim.AdamW([p for p in net.parameters() if p.dim() < 2], lr=1e-3)
    losses = []
    for step in range(steps):
        loss = splat.L1SSIMLoss.apply(net(x, step), target, 0.2)
        muon.zero_grad(set_to_none=True)
        adam.zero_grad(set_to_none=True)
        loss.backward()
        muon.step()
        adam.step()
        losses.append(loss.detach())
        if report and (step % 10 == 0 or step + 1 == steps):
            report("step %4d  loss %.4f" % (step, losses[-1].item()))
    return [float(v) for v in torch.stack(losses).cpu()]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--heads", type=int, default=0, help="of attention between cells; 0: none")
    ap.add_argument("--kv-heads", type=int, help="of keys and values; as many as heads by default")
    ap.add_argument("--dropout", type=float, default=0.0)
    args = ap.parse_args()
    train(args.steps, report=lambda line: print(line, flush=True), heads=args.heads, kv_heads=args.kv_heads,
          dropout=args.dropout)
