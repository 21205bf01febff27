"""A small predictor in front of the splatting layer, trained end to end.

Features of a grid of cells pass through a projection, gated feed-forward
blocks and a head to the raw values of one Gaussian per cell, which are
activated, rendered and compared with target frames; the matrices are trained
by Muon, everything else by AdamW.  Every product, the rendering, the loss and
the optimiser's Newton-Schulz steps run in this package's kernels.

    python examples/fit_predictor.py --steps 60
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_gaussian_splatting_pdr_amd import dense, splat  # noqa: E402


class Predictor(torch.nn.Module):
    """features [B, gx * gy, F] -> frames [B, H, W, C]."""

    def __init__(self, features, width, hidden, blocks, gx, gy, H, W, C, dtype=torch.bfloat16,
                 device="cuda"):
        super().__init__()
        self.grid, self.frame, self.C, self.dtype = (gx, gy), (H, W), C, dtype

        def weight(rows, cols, scale=1.0):
            return torch.nn.Parameter(torch.randn(rows, cols, device=device) * scale * cols ** -0.5)

        self.w_embed = weight(width, features)
        self.b_embed = torch.nn.Parameter(torch.zeros(width, device=device))
        self.w_in = torch.nn.ParameterList(weight(2 * hidden, width) for _ in range(blocks))
        self.w_out = torch.nn.ParameterList(weight(width, hidden, 0.5) for _ in range(blocks))
        self.w_head = weight(5 + C, width, 0.1)
        self.b_head = torch.nn.Parameter(torch.zeros(5 + C, device=device))

    def matrices(self):
        return [p for p in self.parameters() if p.dim() == 2]

    def raw(self, x):
        d = self.dtype
        x = dense.linear(x.to(d), self.w_embed.to(d), self.b_embed.to(d), activation="gelu")
        for w_in, w_out in zip(self.w_in, self.w_out):
            x = dense.gated_mlp(x, w_in.to(d), w_out.to(d), residual=x)
        # the head keeps its sums' 32 bits for the renderer, on top of the grid's own Gaussians
        gx, gy = self.grid
        start = splat.grid_init(x.shape[0], gx, gy, *self.frame, self.C, device=x.device)
        return dense.linear(x, self.w_head.to(d), self.b_head.to(d), residual=start,
                            out_dtype=torch.float32)

    def forward(self, x):
        gx, gy = self.grid
        params = splat.activate(self.raw(x), gx, gy, *self.frame)
        return splat.render(params, *self.frame)


def train(steps=60, B=8, gx=16, gy=16, H=64, W=64, C=3, features=48, width=256, hidden=704,
          blocks=2, seed=0, report=None):
    """Fit frames of a teacher of the same shape; returns the losses."""
    torch.manual_seed(seed)
    net = Predictor(features, width, hidden, blocks, gx, gy, H, W, C)
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
        loss = splat.L1SSIMLoss.apply(net(x), target, 0.2)
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
    train(ap.parse_args().steps, report=lambda line: print(line, flush=True))
