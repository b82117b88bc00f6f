"""Trains two gated, normalised GCN layers on a synthetic partition to reproduce the rows of a fixed
teacher, with quantised halo messages and an AdamW step per epoch.

  python examples/train_nodes.py [--epochs 30] [--state-bits 8]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from quantized_halo_aggregation_amd import synth  # noqa: E402
from quantized_halo_aggregation_amd.pipeline import GpuPartition  # noqa: E402
from quantized_halo_aggregation_amd.training import GatedNormStack  # noqa: E402


def train(epochs: int, state_bits: int, n_in: int = 4000, n_h: int = 1500, nnz: int = 60000, d: int = 64):
    part = synth.make_partition(synth.small_workload(n_in, n_h, nnz, d, bits=("top", 4, 8, 0.1)))
    gp = GpuPartition(part)
    x = torch.from_numpy(part.x).to(gp.device)
    target = GatedNormStack(gp, 2, seed=1).forward(x).clone()
    stack = GatedNormStack(gp, 2, seed=2, state_bits=state_bits)
    losses = []
    for epoch in range(epochs):
        y = stack.step(x, lambda rows: (rows - target) * (2.0 / rows.numel()), lr=1e-2, epoch=epoch)
        losses.append(float((y - target).square().mean()))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--epochs", type=int, default=30)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    args = ap.parse_args()
    for i, loss in enumerate(train(args.epochs, args.state_bits)):
        print(f"epoch {i}: mean squared error {loss:.5f}", flush=True)
