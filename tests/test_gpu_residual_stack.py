"""A training step of deep, residual layers (training.ResidualStack): the residual norms, the gated products, Muon and
AdamW chained with the halo path, against the same chain of float64 oracles, and the example that trains with it."""
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


def _stack(part, **kw):
    from quantized_halo_aggregation_amd.pipeline import GpuPartition
    from quantized_halo_aggregation_amd.training import ResidualStack
    return ResidualStack(GpuPartition(part), **kw)


@pytest.mark.parametrize("norm,matrices", [("rms", "muon"), ("layer", "adamw")])
def test_step_matches_the_chained_oracle(norm, matrices):
    """Raw (32-bit) halo rows, so the whole step is a smooth chain of float64 formulas.  Each of its thirteen stages is
    within a few units of 2^-24 of its own sums of absolute terms; with at most 300 terms a sum, and sums that
    cancel to a tenth of their terms' size, 5e-5 of the largest value bounds rows and gradients."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    part = synth.make_partition(synth.small_workload(900, 300, 9000, 64, bits=("const", 32)))
    H.note(f"residual stack against the oracle, {norm} {matrices}")
    kind = {"rms": B.ROW_RMS, "layer": B.ROW_LAYER}[norm]
    stack = _stack(part, layers=3, norm=kind, matrices=matrices, skip=0.9, branch=0.6, seed=3)
    rng = np.random.default_rng(0)
    for v in [p[k] for p in stack.params for k in ("post_weight", "pre_weight")] + [stack.first_weight]:
        v.copy_(H.dev((1 + 0.2 * rng.standard_normal(64)).astype(np.float32)))
    host = [{k: v.cpu().numpy().astype(np.float64) for k, v in p.items()} for p in stack.params]
    first = stack.first_weight.cpu().numpy().astype(np.float64)
    # forward
    x, kept = part.x.astype(np.float64), []
    u, first_stats = T.row_norm(x, norm, first, None, 1e-6)
    x0 = x
    for p in host:
        a = OA.gcn_aggregate(part.nbr_ptr, part.nbr_idx, part.deg, np.concatenate([u, u[part.mirror]]))
        h, gate, up = T.gated(a, p["w_gate"], p["w_up"], "silu")
        x, u, ps, qs = T.residual_norm(x, h, None, 1, norm, norm, (p["post_weight"], None, p["pre_weight"], None), 0.9, 0.6, 1e-6)
        kept.append((a, h, gate, up, x, ps, qs))
    rows = stack.forward(torch.from_numpy(part.x).cuda())
    H.assert_close_normwise(H.host(rows), u, rtol=5e-5, what="rows")
    # backward
    du, dx, want = part.grad_top.astype(np.float64), None, []
    for p, (a, h, gate, up, x, ps, qs) in zip(reversed(host), reversed(kept)):
        v = (p["post_weight"], None, p["pre_weight"], None)
        dx, dh, _, vec = T.residual_norm_backward(dx, du, x, h, None, 1, norm, norm, v, ps, qs, 0.9, 0.6)
        da, dwg, dwu = T.gated_backward(dh, gate, up, a, p["w_gate"], p["w_up"], "silu")
        cols = OA.gcn_aggregate_t(part.nbr_ptr, part.nbr_idx, part.deg, da)
        du = OA.add_received(cols[:part.n_in], part.mirror, cols[part.n_in:])
        want.insert(0, {"w_gate": dwg, "w_up": dwu, "post_weight": vec[0], "pre_weight": vec[2]})
    dv, dfirst, _ = T.row_norm_backward(du, x0, norm, first_stats, first)
    got = stack.backward(torch.from_numpy(part.grad_top).cuda())
    H.assert_close_normwise(H.host(got), dx + dv, rtol=5e-5, what="dx")
    H.assert_close_normwise(H.host(stack.first_grad), dfirst, rtol=5e-5, what="first weight")
    for l, (grads, ref) in enumerate(zip(stack.grads, want)):
        for k in ref:
            H.assert_close_normwise(H.host(grads[k]), ref[k], rtol=5e-5, what=f"layer {l} {k}")
    # update, from the GPU's own gradients
    before = [{k: H.host(v).astype(np.float64) for k, v in p.items()} for p in stack.params]
    grads = [{k: H.host(v).astype(np.float64) for k, v in p.items()} for p in stack.grads]
    stack.update(1e-2)
    for p, b, g in zip(stack.params, before, grads):
        for k in p:
            if matrices == "muon" and k in ("w_gate", "w_up"):
                five = [(3.4445, -4.7750, 2.0315)] * 5
                ref = T.muon(b[k], g[k], 0 * b[k], 1e-2, 0.95, True, 0.01, 0.2 * 8.0, 1.0, five, 1e-7)[0]
                # lr 0.2 sqrt(64) = 0.016 of O, whose values are off by less than 1e-4, and a rounding of values below 1
                assert np.abs(H.host(p[k]) - ref).max() < 2e-6
            else:
                ref = T.adam_param(b[k], 0.1 * g[k], 0.001 * g[k] * g[k], 1e-2, 0.9, 0.999, 1e-8, 0.01, 1)
                assert np.abs(H.host(p[k]) - ref).max() < 1e-6


def test_replaced_weights_are_the_ones_trained():
    """Weights and gradient buffers put into the layers' dicts (a loaded checkpoint) train as the ones they replace."""
    H.require_gpu()
    import torch
    part = synth.make_partition(synth.small_workload(500, 200, 5000, 32, bits=("const", 32)))
    x, grad = torch.from_numpy(part.x).cuda(), torch.from_numpy(part.grad_top).cuda()
    H.note("residual stack with replaced weights")
    stacks = [_stack(part, layers=2, seed=5) for _ in range(2)]
    old = stacks[1].params[0]["w_gate"]
    kept = old.clone()
    for d in stacks[1].params + stacks[1].grads:
        for k in d:
            d[k] = d[k].clone()
    stacks[1].first_weight = stacks[1].first_weight.clone()
    for _ in range(2):
        for s in stacks:
            s.step(x, lambda y: grad, 1e-2)
    for a, b in zip(*(s.params for s in stacks)):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    assert torch.equal(stacks[0].first_weight, stacks[1].first_weight)
    assert torch.equal(old, kept) and not torch.equal(stacks[1].params[0]["w_gate"], kept)


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_runs(bits):
    H.require_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_nodes
    H.note(f"residual training example, {bits}-bit moments")
    losses = train_nodes.train(10, bits, n_in=1200, n_h=400, nnz=15000, d=32, residual=True)
    assert len(losses) == 10 and np.isfinite(losses).all()


def test_a_captured_step_replays():
    """Forward, backward and both optimisers' steps in one graph: four replays against as many eager steps."""
    H.require_gpu()
    import torch
    part = synth.make_partition(synth.small_workload(700, 250, 8000, 32, bits=("const", 32)))
    x, grad = torch.from_numpy(part.x).cuda(), torch.from_numpy(part.grad_top).cuda()
    H.note("residual stack captured")
    eager, stack = (_stack(part, layers=3, seed=7) for _ in range(2))
    for s in (eager, stack):                    # a first step outside of the graph, as a program's warm-up
        s.step(x, lambda y: grad, 1e-2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows = stack.forward(x)
        stack.backward(grad)
        stack.muon.step(stack._of(stack.grads, stack._matrices), 1e-2)
    for turn in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = eager.forward(x)
        eager.backward(grad)
        eager.muon.step(eager._of(eager.grads, eager._matrices), 1e-2)
        assert torch.equal(rows, want), turn
        for a, b in zip(stack.params + stack.grads, eager.params + eager.grads):
            assert all(torch.equal(a[k], b[k]) for k in a), turn
        x.mul_(1.01)


def test_refusals():
    H.require_gpu()
    from quantized_halo_aggregation_amd import binding as B
    part = synth.make_partition(synth.small_workload(300, 100, 3000, 32, bits=("const", 32)))
    for bad in (dict(layers=0), dict(layers=2, norm=B.ROW_NONE), dict(layers=2, matrices="sgd")):
        with pytest.raises(ValueError):
            _stack(part, **bad)
