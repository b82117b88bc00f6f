"""A training step of gated, normalised GCN layers on one partition: the halo path of pipeline.py with
the gated projection, the group norm and the optimiser in place of the plain projection.

  forward   quantize_pack(send set) -> [exchange] -> dequant_aggregate_fwd -> gated_project
            -> group_norm_fwd (per node, with its activation)
  backward  group_norm_bwd -> gated_backward -> aggregate_bwd_quantize (every column: inner rows stored, halo
            rows coded) -> [exchange] -> dequant_aggregate_fwd over the mirror map (received gradients added)
  update    adamw_step over every layer's W_gate, W_up, norm weight and norm bias

and of deep stacks of the same layers around a residual stream (ResidualStack), whose blocks have a norm before and
one after them and whose matrices take orthogonalised updates:

  forward   residual_norm_fwd (the first norm) -> per layer quantize_pack -> [exchange] -> dequant_aggregate_fwd ->
            gated_project -> residual_norm_fwd (the norm after the block, the stream, the next block's norm)
  backward  residual_norm_bwd -> gated_backward -> aggregate_bwd_quantize -> [exchange] -> dequant_aggregate_fwd
  update    muon_step over every layer's W_gate and W_up, adamw_step over the norms' weights

Everything numeric runs in libqha's kernels on the current stream; this module lays out buffers and
issues the calls in order.
"""
from __future__ import annotations

import torch

from . import binding as B
from . import pipeline

NAMES = ("w_gate", "w_up", "norm_weight", "norm_bias")


def _take_rows(held, x):
    """Copies x into `held`; rows that a copy would broadcast are refused."""
    if x.shape != held.shape:
        raise ValueError(f"x must be {held.shape[0]} x {held.shape[1]}, got {tuple(x.shape)}")
    held.copy_(x)


class GatedNormStack:
    """`layers` layers of width gp.d on a GCN partition, their gradients and an AdamW optimiser.

    Layer l: A = aggregate(X_l, halo messages), H = act(A W_gate^T) * (A W_up^T), X_{l+1} =
    norm_act(group_norm(H)).  forward() returns the last layer's rows, backward() takes their gradient and
    leaves the parameters' in self.grads, update() takes the optimiser's step; step() does the three."""

    def __init__(self, gp: pipeline.GpuPartition, layers: int, n_groups: int = 8, act: int = B.ACT_SILU,
                 norm_act: int = B.ACT_NONE, state_bits: int = 32, weight_decay: float = 0.01, seed: int = 0):
        if gp.model != "gcn":
            raise ValueError("the stack aggregates as a GCN")
        if layers < 1 or gp.d % n_groups:
            raise ValueError(f"{layers} layers of {gp.d} channels in {n_groups} groups")
        self.gp, self.layers, self.n_groups, self.act, self.norm_act = gp, layers, n_groups, act, norm_act
        dev, n, d = gp.device, gp.n_in, gp.d
        gen = torch.Generator(device="cpu").manual_seed(seed)
        draw = lambda: (torch.randn(d, d, generator=gen) * d ** -0.5).to(dev)
        self.params = [{"w_gate": draw(), "w_up": draw(), "norm_weight": torch.ones(d, device=dev),
                        "norm_bias": torch.zeros(d, device=dev)} for _ in range(layers)]
        self.grads = [{k: torch.empty_like(v) for k, v in p.items()} for p in self.params]
        self.opt = B.AdamW([p[k] for p in self.params for k in NAMES], bits=state_bits, weight_decay=weight_decay)
        rows = lambda: torch.empty(n, d, dtype=torch.float32, device=dev)
        # kept for the backward, per layer: A, gate, up, H and the norm's statistics
        self.X = [rows() for _ in range(layers + 1)]
        self.A, self.gate, self.up, self.H = ([rows() for _ in range(layers)] for _ in range(4))
        self.mean, self.rstd = ([torch.empty(n, n_groups, device=dev) for _ in range(layers)] for _ in range(2))
        self.dX, self.dH = [rows(), rows()], rows()
        self.msg_f, self.msg_b = gp.new_messages(), gp.new_messages()
        need = max(B.gated_project_workspace(torch.float32, n, d, d), B.gated_backward_workspace(torch.float32, n, d, d),
                   *(B.group_norm_workspace(n, 1, d, n_groups, b) for b in (False, True)), 16)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def forward(self, x, epoch: int = 0):
        """The last layer's rows for the inner rows x [n_in, d] (halo rows quantised at the partition's
        widths)."""
        gp = self.gp
        _take_rows(self.X[0], x)
        for l, p in enumerate(self.params):
            gp.quantize_send(self.X[l], gp.mirror, self.msg_f, epoch, 2 * l)
            gp.aggregate_fwd(self.X[l], self.msg_f, self.A[l])
            B.gated_project(self.A[l], p["w_gate"], p["w_up"], self.H[l], gate=self.gate[l], up=self.up[l], act=self.act,
                            workspace=self.ws)
            B.group_norm_fwd(self.H[l], self.X[l + 1], self.n_groups, weight=p["norm_weight"], bias=p["norm_bias"],
                             mean=self.mean[l], rstd=self.rstd[l], act=self.norm_act, workspace=self.ws)
        return self.X[-1]

    def backward(self, grad_out, epoch: int = 0):
        """Gradients of every parameter, from grad_out [n_in, d] and the last forward; returns that of x."""
        gp, g = self.gp, grad_out
        for l in reversed(range(self.layers)):
            p, dp = self.params[l], self.grads[l]
            B.group_norm_bwd(g, self.H[l], self.mean[l], self.rstd[l], self.dH, self.n_groups, weight=p["norm_weight"],
                             bias=p["norm_bias"], dweight=dp["norm_weight"], dbias=dp["norm_bias"], act=self.norm_act,
                             workspace=self.ws)
            da, g = self.dX[0], self.dX[1]
            B.gated_backward(self.dH, self.gate[l], self.up[l], self.A[l], p["w_gate"], p["w_up"], da, dp["w_gate"],
                             dp["w_up"], act=self.act, workspace=self.ws)
            gp.aggregate_bwd_all_quantize(da, g, self.msg_b, epoch, 2 * l + 1, 0)
            gp.add_received(self.msg_b, g)
        return g

    def update(self, lr: float):
        # as they are now: a caller may have put other tensors in their places
        self.opt.params = [p[k] for p in self.params for k in NAMES]
        self.opt.step([g[k] for g in self.grads for k in NAMES], lr)

    def step(self, x, loss_grad, lr: float, epoch: int = 0):
        """One training step; loss_grad maps the last layer's rows to their gradient.  Returns the rows."""
        y = self.forward(x, epoch)
        self.backward(loss_grad(y), epoch)
        self.update(lr)
        return y


class ResidualStack:
    """`layers` gated layers of width gp.d around a residual stream on a GCN partition, and their optimisers.

    X_0 = x, U_0 = norm(X_0); layer l: A = aggregate(U_l, halo messages of U_l), H = act(A W_gate^T) * (A W_up^T),
    X_{l+1} = skip X_l + branch norm(H), U_{l+1} = norm(X_{l+1}), every norm a row's (norm, an RMS or a layer norm)
    with a weight per channel.  forward() returns U_layers, backward() takes its gradient and leaves the
    parameters' in self.grads and self.first_grad, update() takes the optimisers' steps; step() does the three.  Layer
    l's dict holds w_gate, w_up, post_weight (of the norm of H) and pre_weight (of X_{l+1}); first_weight is X_0's.

    matrices="muon" gives W_gate and W_up to B.Muon and the norms' weights to B.AdamW, "adamw" all of them."""

    def __init__(self, gp: pipeline.GpuPartition, layers: int, act: int = B.ACT_SILU, norm: int = B.ROW_RMS,
                 skip: float = 1.0, branch: float = 1.0, eps: float = 1e-6, matrices: str = "muon", state_bits: int = 32,
                 weight_decay: float = 0.01, seed: int = 0):
        if gp.model != "gcn":
            raise ValueError("the stack aggregates as a GCN")
        if layers < 1 or norm not in (B.ROW_RMS, B.ROW_LAYER) or matrices not in ("muon", "adamw"):
            raise ValueError(f"{layers} layers, norm {norm}, matrices by {matrices!r}")
        self.gp, self.layers, self.act, self.norm = gp, layers, act, norm
        self.skip, self.branch, self.eps = skip, branch, eps
        dev, n, d = gp.device, gp.n_in, gp.d
        gen = torch.Generator(device="cpu").manual_seed(seed)
        draw = lambda: (torch.randn(d, d, generator=gen) * d ** -0.5).to(dev)
        one = lambda: torch.ones(d, device=dev)
        self.params = [{"w_gate": draw(), "w_up": draw(), "post_weight": one(), "pre_weight": one()} for _ in range(layers)]
        self.grads = [{k: torch.empty_like(v) for k, v in p.items()} for p in self.params]
        self.first_weight, self.first_grad = one(), torch.empty(d, device=dev)
        self._matrices = ("w_gate", "w_up") if matrices == "muon" else ()
        self._vectors = ("post_weight", "pre_weight") if matrices == "muon" else ("w_gate", "w_up", "post_weight", "pre_weight")
        self.muon = B.Muon(self._of(self.params, self._matrices), weight_decay=weight_decay, scale="rms")
        self.adamw = B.AdamW(self._of(self.params, self._vectors) + [self.first_weight], bits=state_bits,
                             weight_decay=weight_decay)
        rows = lambda: torch.empty(n, d, dtype=torch.float32, device=dev)
        # kept for the backward: the stream and, per layer, A, gate, up, H and the norms' statistics
        self.X, self.U = [rows() for _ in range(layers + 1)], rows()
        self.A, self.gate, self.up, self.H = ([rows() for _ in range(layers)] for _ in range(4))
        self.post_stats = [torch.empty(n, 2, device=dev) for _ in range(layers)]
        self.pre_stats = [torch.empty(n, 2, device=dev) for _ in range(layers + 1)]
        self.dX, self.dU, self.dA, self.dH = rows(), rows(), rows(), rows()
        self.msg_f, self.msg_b = gp.new_messages(), gp.new_messages()
        need = max(B.gated_project_workspace(torch.float32, n, d, d), B.gated_backward_workspace(torch.float32, n, d, d),
                   B.residual_norm_workspace(n, d), 16)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

    @staticmethod
    def _of(dicts, names):
        return [p[k] for p in dicts for k in names]

    def forward(self, x, epoch: int = 0):
        """The last layer's normalised rows for the inner rows x [n_in, d] (halo rows quantised at the
        partition's widths)."""
        gp = self.gp
        _take_rows(self.X[0], x)
        B.residual_norm_fwd(self.X[0], None, None, self.U, post=B.ROW_NONE, pre=self.norm, pre_weight=self.first_weight,
                            eps=self.eps, pre_stats=self.pre_stats[0])
        for l, p in enumerate(self.params):
            gp.quantize_send(self.U, gp.mirror, self.msg_f, epoch, 2 * l)
            gp.aggregate_fwd(self.U, self.msg_f, self.A[l])
            B.gated_project(self.A[l], p["w_gate"], p["w_up"], self.H[l], gate=self.gate[l], up=self.up[l], act=self.act,
                            workspace=self.ws)
            B.residual_norm_fwd(self.X[l], self.H[l], self.X[l + 1], self.U, post=self.norm, pre=self.norm,
                                post_weight=p["post_weight"], pre_weight=p["pre_weight"], skip=self.skip,
                                branch=self.branch, eps=self.eps, post_stats=self.post_stats[l],
                                pre_stats=self.pre_stats[l + 1])
        return self.U

    def backward(self, grad_out, epoch: int = 0):
        """Gradients of every parameter, from grad_out [n_in, d] and the last forward; returns that of x."""
        gp, du, dx = self.gp, grad_out, None
        for l in reversed(range(self.layers)):
            p, dp = self.params[l], self.grads[l]
            B.residual_norm_bwd(dx, du, self.X[l + 1], self.H[l], self.dX, self.dH, post=self.norm, pre=self.norm,
                                post_stats=self.post_stats[l], pre_stats=self.pre_stats[l + 1],
                                post_weight=p["post_weight"], pre_weight=p["pre_weight"], skip=self.skip,
                                branch=self.branch, dpost_weight=dp["post_weight"], dpre_weight=dp["pre_weight"],
                                workspace=self.ws)
            B.gated_backward(self.dH, self.gate[l], self.up[l], self.A[l], p["w_gate"], p["w_up"], self.dA, dp["w_gate"],
                             dp["w_up"], act=self.act, workspace=self.ws)
            gp.aggregate_bwd_all_quantize(self.dA, self.dU, self.msg_b, epoch, 2 * l + 1, 0)
            gp.add_received(self.msg_b, self.dU)
            du, dx = self.dU, self.dX
        B.residual_norm_bwd(dx, du, self.X[0], None, self.dX, None, post=B.ROW_NONE, pre=self.norm,
                            pre_stats=self.pre_stats[0], pre_weight=self.first_weight, dpre_weight=self.first_grad,
                            workspace=self.ws)
        return self.dX

    def update(self, lr: float):
        """Muon's updates of matrices have AdamW's size (scale="rms"), so that both take one learning rate."""
        # as they are now: a caller may have put other tensors in their places
        self.muon.params = self._of(self.params, self._matrices)
        self.adamw.params = self._of(self.params, self._vectors) + [self.first_weight]
        self.muon.step(self._of(self.grads, self._matrices), lr)
        self.adamw.step(self._of(self.grads, self._vectors) + [self.first_grad], lr)

    def step(self, x, loss_grad, lr: float, epoch: int = 0):
        """One training step; loss_grad maps the last layer's rows to their gradient.  Returns the rows."""
        y = self.forward(x, epoch)
        self.backward(loss_grad(y), epoch)
        self.update(lr)
        return y
