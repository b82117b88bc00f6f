"""A training step of gated, normalised layers (training.GatedNormStack): the operators chained with the
halo path, against the same chain of float64 oracles, and the example that trains with it."""
import os
import sys

import numpy as np
import pytest

import gpu_helpers as H
from oracle import aggregate as OA
from oracle import train as T
from quantized_halo_aggregation_amd import synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_step_matches_the_chained_oracle():
    """Raw (32-bit) halo rows, so the whole step is a smooth chain of float64 formulas.  Each of its eight stages
    is within a few units of 2^-24 of its own sums of absolute terms; with at most 300 terms a sum, and sums that
    cancel to a tenth of their terms' size, 2e-5 of the largest value bounds rows and gradients."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd.pipeline import GpuPartition
    from quantized_halo_aggregation_amd.training import GatedNormStack
    part = synth.make_partition(synth.small_workload(900, 300, 9000, 64, bits=("const", 32)))
    gp = GpuPartition(part)
    H.note("training step against the oracle")
    stack = GatedNormStack(gp, 2, n_groups=4, norm_act=2, seed=3)
    rng = np.random.default_rng(0)
    for p in stack.params:
        p["norm_weight"].copy_(H.dev((1 + 0.2 * rng.standard_normal(64)).astype(np.float32)))
        p["norm_bias"].copy_(H.dev((0.2 * rng.standard_normal(64)).astype(np.float32)))
    host = [{k: v.cpu().numpy().astype(np.float64) for k, v in p.items()} for p in stack.params]
    grad = part.grad_top.astype(np.float64)
    # forward
    x, kept = part.x.astype(np.float64), []
    for p in host:
        a = OA.gcn_aggregate(part.nbr_ptr, part.nbr_idx, part.deg, np.concatenate([x, x[part.mirror]]))
        h, gate, up = T.gated(a, p["w_gate"], p["w_up"], "silu")
        y, mean, rstd = T.group_norm(h, p["norm_weight"], p["norm_bias"], 4, 1, 1e-5, "silu")
        kept.append((a, h, gate, up, mean, rstd))
        x = y
    rows = stack.forward(torch.from_numpy(part.x).cuda())
    H.assert_close_normwise(H.host(rows), x, rtol=2e-5, what="rows")
    # backward
    g, want = grad, []
    for p, (a, h, gate, up, mean, rstd) in zip(reversed(host), reversed(kept)):
        dh, dw, db = T.group_norm_backward(g, h, mean, rstd, p["norm_weight"], p["norm_bias"], 4, 1, "silu")
        da, dwg, dwu = T.gated_backward(dh, gate, up, a, p["w_gate"], p["w_up"], "silu")
        cols = OA.gcn_aggregate_t(part.nbr_ptr, part.nbr_idx, part.deg, da)
        g = OA.add_received(cols[:part.n_in], part.mirror, cols[part.n_in:])
        want.insert(0, {"w_gate": dwg, "w_up": dwu, "norm_weight": dw, "norm_bias": db})
    dx = stack.backward(torch.from_numpy(part.grad_top).cuda())
    H.assert_close_normwise(H.host(dx), g, rtol=2e-5, what="dx")
    for l, (got, ref) in enumerate(zip(stack.grads, want)):
        for k in ref:
            H.assert_close_normwise(H.host(got[k]), ref[k], rtol=2e-5, what=f"layer {l} {k}")
    # update, from the GPU's own gradients: one first step moves every weight by lr against its gradient's sign
    before = [H.host(stack.params[0][k]).copy() for k in ("w_gate", "norm_bias")]
    stack.update(1e-2)
    for k, old in zip(("w_gate", "norm_bias"), before):
        gk = H.host(stack.grads[0][k]).astype(np.float64)
        step = T.adam_param(old, 0.1 * gk, 0.001 * gk * gk, 1e-2, 0.9, 0.999, 1e-8, 0.01, 1)
        assert np.abs(H.host(stack.params[0][k]) - step).max() < 1e-6


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_learns(bits):
    H.require_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_nodes
    H.note(f"training example, {bits}-bit moments")
    losses = train_nodes.train(25, bits, n_in=1200, n_h=400, nnz=15000, d=32)
    assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0], losses[::6]


def test_replaced_weights_are_the_ones_trained():
    """Weights and gradient buffers put into the layers' dicts (a loaded checkpoint) train as the ones they replace."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd.pipeline import GpuPartition
    from quantized_halo_aggregation_amd.training import GatedNormStack
    part = synth.make_partition(synth.small_workload(500, 200, 5000, 32, bits=("const", 32)))
    gp = GpuPartition(part)
    x, grad = torch.from_numpy(part.x).cuda(), torch.from_numpy(part.grad_top).cuda()
    H.note("training step with replaced weights")
    stacks = [GatedNormStack(gp, 2, seed=5) for _ in range(2)]
    old = stacks[1].params[0]["w_gate"]
    kept = old.clone()
    for d in stacks[1].params + stacks[1].grads:
        for k in d:
            d[k] = d[k].clone()
    for _ in range(2):
        for s in stacks:
            s.step(x, lambda y: grad, 1e-2)
    for a, b in zip(*(s.params for s in stacks)):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    assert torch.equal(old, kept) and not torch.equal(stacks[1].params[0]["w_gate"], kept)
