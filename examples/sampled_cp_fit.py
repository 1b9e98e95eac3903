"""Fit a CP model to sampled entries of a tensor by clipped stochastic gradient steps.

For tensors that are only partly observed, or too large to sweep (CP-ALS reads every
entry in every sweep): each step takes a batch of (coordinates, value) pairs and uses

    cp_entries        the model's values at the coordinates,
    cp_entries_grad   the squared error's gradient for every factor,
    embedding         the rows of a factor that the batch touched, scaled by a penalty,
    embedding_grad    which are added to that factor's gradient, row by row,
    clip_grad_norm    all gradients, scaled so that their common norm is at most a limit,
    orthogonal_step   (--orthogonal) momentum and the update along the orthogonal matrix
                      nearest to it, instead of along the momentum itself.

Nothing in a step waits for the GPU.

    python examples/sampled_cp_fit.py --dims 60 50 40 --rank 8 --steps 1500
    python examples/sampled_cp_fit.py --orthogonal
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_tensor_decomposition_gb300 as mk  # noqa: E402


def gradients(factors, coords, values, penalty: float = 0.0, max_norm: float | None = None):
    """Mean squared error of a batch, the gradients of
        mean over samples of (x_s - y_s)^2 + penalty * sum over n of |A_n(c_sn, :)|^2
    for every factor, clipped to max_norm, and their norm before clipping."""
    S = coords.shape[0]
    residual = mk.cp_entries(factors, coords) - values
    grads = mk.cp_entries_grad(factors, coords, residual * (2.0 / S))
    if penalty > 0.0:
        for n, (A, G) in enumerate(zip(factors, grads)):
            rows = mk.embedding(A, coords[:, n], scale=2.0 * penalty / S)
            mk.embedding_grad(coords[:, n], rows, A.shape[0], out=G, accumulate=True)
    norm = mk.grad_norm(grads) if max_norm is None else mk.clip_grad_norm(grads, max_norm)
    return residual.square().mean(), grads, norm


def fit(coords, values, dims, rank: int, steps: int, batch: int, rate: float = 0.3, momentum: float = 0.9,
        penalty: float = 1e-4, max_norm: float = 1.0, seed: int = 0, orthogonal: bool = False):
    """Factors (list of dims[n] x rank, float32) after `steps` steps over random batches of
    the samples, and the batches' mean squared errors.  orthogonal: every factor moves along its
    orthogonalised momentum, all singular directions alike, by `rate`."""
    gen = torch.Generator(device=coords.device).manual_seed(seed)
    factors = [torch.randn(n, rank, generator=gen, device=coords.device).mul_(0.3) for n in dims]
    velocity = [torch.zeros_like(a) for a in factors]
    losses = []
    for _ in range(steps):
        pick = torch.randint(coords.shape[0], (batch,), generator=gen, device=coords.device)
        loss, grads, _ = gradients(factors, coords[pick], values[pick], penalty, max_norm)
        if orthogonal:
            mk.orthogonal_step(factors, grads, velocity, rate, momentum=momentum, scale=1.0)
        else:
            for A, V, G in zip(factors, velocity, grads):
                V.mul_(momentum).add_(G)
                A.sub_(V, alpha=rate)
        losses.append(loss)
    return factors, torch.stack(losses)


def samples(dims, rank: int, count: int, seed: int = 1, noise: float = 0.01):
    """Entries of a random rank-`rank` tensor of unit variance, at random coordinates."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    factors = [torch.randn(n, rank, generator=gen, device="cuda") for n in dims]
    coords = torch.stack([torch.randint(n, (count,), generator=gen, device="cuda", dtype=torch.int32)
                          for n in dims], dim=1)
    values = mk.cp_entries(factors, coords)
    scale = values.square().mean().sqrt()
    return coords, values / scale + noise * torch.randn(count, generator=gen, device="cuda")


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dims", type=int, nargs="+", default=[60, 50, 40])
    ap.add_argument("--rank", type=int, default=8)
    ap.add_argument("--samples", type=int, default=60000)
    ap.add_argument("--batch", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=1500)
    ap.add_argument("--orthogonal", action="store_true")
    args = ap.parse_args()
    coords, values = samples(args.dims, args.rank, args.samples)
    _, losses = fit(coords, values, args.dims, 2 * args.rank, args.steps, args.batch,
                    rate=0.02 if args.orthogonal else 1.0, orthogonal=args.orthogonal)
    every = max(1, args.steps // 10)
    for k in range(0, args.steps, every):
        print(f"step {k:5d}: mean squared error {float(losses[k]):.5f}")
    print(f"last {every} steps: {float(losses[-every:].mean()):.5f}")


if __name__ == "__main__":
    main()
