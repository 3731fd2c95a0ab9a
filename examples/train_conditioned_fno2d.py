"""Train a residual FNO2d conditioned on time: the solution of the heat equation
on a periodic square, a(x) and tau in, exp(tau Laplacian) a out.

    python examples/train_conditioned_fno2d.py --steps 200

Every field operation of the step runs in the library: the lift and projection and
each block's 1x1 convolution (channel_mix, inputs kept in 8 bits), its
spectral convolution (spectral_conv, retained spectra kept), and the norms before
and after it with the gate that carries the condition and the learned residual
scale (norm_residual, fields kept in 8 bits). Data and weights are synthetic.
"""

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spectral_convolution_amd as fno  # noqa: E402
from workloads.generate import gaussian_random_field  # noqa: E402

TAU = 2e-3  # longest diffusion time; the square has side 1


def heat_batch(rng, batch, grid):
    """(a, tau, solution): float64 fields [batch][1][H][W], tau [batch] in [0, 1]."""
    a = gaussian_random_field(rng, (batch, 1), grid)
    tau = rng.uniform(size=batch)
    k = [2 * math.pi * np.fft.fftfreq(n, 1.0 / n) for n in grid]
    k2 = k[0][:, None] ** 2 + k[1][None, :] ** 2
    decay = np.exp(-TAU * tau[:, None, None, None] * k2)
    return a, tau, np.fft.ifft2(np.fft.fft2(a) * decay).real


class ConditionedFno2d(torch.nn.Module):
    """x_0 = lift(features); per block v = GELU(W u + b + spectral(u)),
    x += scale gate(tau) N(v), u = N'(x); out = projection(u)."""

    def __init__(self, batch, grid, channels=32, modes=(12, 12), blocks=4, hidden=64, keep="8bit", device=0):
        super().__init__()
        g = torch.Generator().manual_seed(0)

        def param(*shape, bound=None, value=None):
            t = torch.full(shape, float(value)) if bound is None else torch.rand(shape, generator=g).mul_(2).sub_(1).mul_(bound)
            return torch.nn.Parameter(t.to(f"cuda:{device}"))

        self.keep = keep
        self.plan = fno.fno_plan_create(2, batch, channels, channels, grid, modes, "f32", device)
        c = channels
        self.lift, self.lift_bias = param(c, 3, bound=3 ** -0.5), param(c, bound=3 ** -0.5)
        self.blocks = torch.nn.ModuleList()
        for _ in range(blocks):
            b = torch.nn.Module()
            shape = self.plan.split_shape()
            b.wr, b.wi = param(*shape, bound=1 / c), param(*shape, bound=1 / c)
            b.w, b.bias = param(c, c, bound=c ** -0.5), param(c, bound=c ** -0.5)
            b.w_post, b.b_post, b.w_pre, b.b_pre = param(c, value=1), param(c, value=0), param(c, value=1), param(c, value=0)
            b.scale = param(c, value=0.3)
            b.cond, b.cond_bias = param(c, bound=0.1), param(c, value=1)
            self.blocks.append(b)
        self.q1, self.q1_bias = param(hidden, c, bound=c ** -0.5), param(hidden, bound=c ** -0.5)
        self.q2, self.q2_bias = param(1, hidden, bound=hidden ** -0.5), param(1, bound=hidden ** -0.5)

    def forward(self, features, tau):
        x = fno.channel_mix(features, self.lift, self.lift_bias)
        u = x
        for b in self.blocks:
            v = fno.channel_mix(u, b.w, b.bias, fno.spectral_conv(self.plan, u, b.wr, b.wi), act=1)
            gate = tau[:, None] * b.cond + b.cond_bias
            norm = fno.NormParams("layer", 1e-5, b.w_post, b.b_post, gate, b.scale, b.w_pre, b.b_pre)
            x, u = fno.norm_residual(x, v, norm, keep=self.keep)
        return fno.channel_mix(fno.channel_mix(u, self.q1, self.q1_bias, act=1), self.q2, self.q2_bias)

    def close(self):
        fno.fno_plan_destroy(self.plan)


def train(steps=100, batch=16, grid=(64, 64), channels=32, modes=(12, 12), blocks=4, lr=2e-3, keep="8bit", device=0,
          report=None):
    """The relative L2 losses of `steps` Adam steps on fresh samples."""
    rng = np.random.default_rng(0)
    dev = f"cuda:{device}"
    net = ConditionedFno2d(batch, grid, channels, modes, blocks, keep=keep, device=device)
    opt = torch.optim.Adam(net.parameters(), lr=lr)
    xy = np.broadcast_to(np.stack(np.meshgrid(*[np.arange(n) / n for n in grid], indexing="ij")), (batch, 2) + grid)
    losses = []
    try:
        for step in range(steps):
            a, tau, want = heat_batch(rng, batch, grid)
            to = lambda t: torch.from_numpy(np.ascontiguousarray(t)).float().to(dev)  # noqa: E731
            features, tau, want = to(np.concatenate([a, xy], 1)), to(tau), to(want)
            opt.zero_grad(set_to_none=True)
            loss = (net(features, tau) - want).norm() / want.norm()
            loss.backward()
            opt.step()
            losses.append(loss.item())
            if report and (step % report == 0 or step == steps - 1):
                print(f"step {step}: relative L2 {losses[-1]:.4f}, "
                      f"peak {torch.cuda.max_memory_allocated(device) / 2 ** 20:.0f} MiB", flush=True)
        torch.cuda.synchronize(device)
    finally:
        net.close()
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--size", type=int, default=64, help="grid points a side")
    ap.add_argument("--channels", type=int, default=32)
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--keep", choices=("8bit", "whole"), default="8bit", help="how the norms keep their fields")
    a = ap.parse_args(argv)
    train(a.steps, a.batch, (a.size, a.size), a.channels, blocks=a.blocks, keep=a.keep, report=max(1, a.steps // 10))


if __name__ == "__main__":
    main()
