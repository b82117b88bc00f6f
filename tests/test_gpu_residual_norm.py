"""qha_residual_norm_fwd and qha_residual_norm_bwd against the float64 oracle.

Tolerances count roundings, u = 2^-24 the unit roundoff of float32, and half a step of the output's type.  A float32
sum over a row passes at most K = 48 additions (32 in a thread, 6 between lanes, 8 between wavefronts, 2 to spare).
Forward: a mean is off by K u mean|v|; 1 / deviation by (K / 2 + 6) u of itself (the mean's error cancels to first
order); so xhat is off by eh = u (K rstd mean|v| + 2 rstd (|v| + |mean|) + (K / 2 + 6) |xhat|), z by |w| eh + 3 u (|z| + |b|),
x' by |branch g| of that + 4 u (|skip x| + |branch g z|).  u's norm sees an x' that is off by at most E in its row, which
moves xhat' by at most rstd E (2 + |xhat'|), and adds an eh of its own.  Backward, with given statistics: the gradient
through a norm is rstd (q - mean q - xhat mean(q xhat)), off by (K + 10) u rstd (|q| + mean|q| + |xhat| mean|q xhat|) and by the same
form of its input's error.  Sums over rows run over at most rows / 256 + 1 terms in float32 (256 teams or more share them out)
and 20 more additions, then in float64.
"""
import numpy as np
import pytest

import gpu_helpers as H
from oracle import train as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
K = 48
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 0.0, "bfloat16": 0.0, "float16": 2.0 ** -25}      # half a step of subnormals
TYPES = [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float16"), ("float32", "bfloat16"),
         ("float32", "float16")]                                     # the stream's, the branch's
KINDS = ["none", "rms", "layer"]

# rows, positions, channels: every team size and vector count, short last vectors, one row to many
SHAPES = [(1, 1, 8), (5, 5, 16), (33, 1, 40), (291, 97, 64), (1001, 1, 128), (64, 2, 136), (77, 7, 256), (3001, 3001, 96),
          (130, 1, 512), (12, 4, 520), (9, 1, 1024), (8, 8, 1032), (300, 1, 2048), (21, 3, 2056), (6, 2, 4096), (5, 1, 4104),
          (3, 3, 8192), (700, 350, 8192), (40000, 1, 32), (600, 1, 1000)]


def _t(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(getattr(torch, dtype)).cuda()


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


class Case:
    """Inputs of both directions, and what the oracle says of them."""

    def __init__(self, shape, types, post, pre, gate=True, bias=True, weight=True, block=True, dy=True, skip=0.9, branch=1.3,
                 seed=5, shift=0.3):
        rng = np.random.default_rng(seed)
        self.rows, self.positions, self.c = shape
        self.stream, self.type = types
        self.post, self.pre, self.skip, self.branch, self.eps = post, pre, np.float32(skip), np.float32(branch), 1e-5
        if not block:
            self.skip, self.branch = np.float32(1), np.float32(1)
        n, c = self.rows, self.c
        draw = lambda s, *sh: rng.standard_normal(sh) * s
        self.x = _t(draw(1.5, n, c) + shift, self.stream)
        self.h = _t(draw(0.8, n, c) + shift, self.type) if block else None
        self.gate = _t(0.5 + draw(0.5, n // self.positions, c), self.type) if gate and block else None
        vec = lambda mid, on: _t(mid + draw(0.3, c), "float32") if on else None
        self.vectors = [vec(1, weight and block), vec(0, bias and block), vec(1, weight and pre != "none"),
                        vec(0, bias and pre != "none")]
        self.dy = _t(draw(1, n, c), self.stream) if dy or pre == "none" else None
        self.du = _t(draw(1, n, c), self.type) if pre != "none" else None

    def kinds(self):
        from quantized_halo_aggregation_amd import binding as B
        k = {"none": B.ROW_NONE, "rms": B.ROW_RMS, "layer": B.ROW_LAYER}
        return dict(post=k[self.post], pre=k[self.pre], post_weight=self.vectors[0], post_bias=self.vectors[1],
                    pre_weight=self.vectors[2], pre_bias=self.vectors[3], gate=self.gate, positions=self.positions,
                    skip=float(self.skip), branch=float(self.branch))

    def new(self, dtype, *shape):
        import torch
        return torch.full(shape, float("nan"), dtype=getattr(torch, dtype), device="cuda")

    def run_fwd(self, **over):
        from quantized_halo_aggregation_amd import binding as B
        n, c = self.rows, self.c
        block, pre = self.h is not None, self.pre != "none"
        out = dict(y=self.new(self.stream, n, c) if block else None, u=self.new(self.type, n, c) if pre else None,
                   post_stats=self.new("float32", n, 2) if block and self.post != "none" else None,
                   pre_stats=self.new("float32", n, 2) if pre else None)
        out.update(over)
        B.residual_norm_fwd(self.x, self.h, out["y"], out["u"], post_stats=out["post_stats"], pre_stats=out["pre_stats"],
                            eps=self.eps, **self.kinds())
        return out

    def kept(self):
        """The stream and statistics that a backward is given: the oracle's, rounded to what the forward stores."""
        v = [_np(t) for t in self.vectors]
        y, _, ps, _ = T.residual_norm(_np(self.x), _np(self.h), _np(self.gate), self.positions, self.post, self.pre, v,
                                      self.skip, self.branch, self.eps)
        self.y = _t(y, self.stream)
        self.post_stats = _t(ps, "float32") if ps is not None and self.post != "none" else None
        self.pre_stats = _t(T.row_norm(_np(self.y), self.pre, None, None, self.eps)[1], "float32") if self.pre != "none" else None

    def run_bwd(self, **over):
        import torch
        from quantized_halo_aggregation_amd import binding as B
        n, c = self.rows, self.c
        block = self.h is not None
        out = dict(dx=self.new(self.stream, n, c), dh=self.new(self.type, n, c) if block else None,
                   dgate=self.new(self.type, n // self.positions, c) if self.gate is not None else None,
                   vectors=[self.new("float32", c) if on else None for on in (block, block, self.pre != "none", self.pre != "none")])
        out.update(over)
        ws = torch.empty(max(B.residual_norm_workspace(n, c, self.positions), 16), dtype=torch.uint8, device="cuda")
        v = out["vectors"]
        B.residual_norm_bwd(self.dy, self.du, self.y, self.h, out["dx"], out["dh"], post_stats=self.post_stats,
                            pre_stats=self.pre_stats, dgate=out["dgate"], dpost_weight=v[0], dpost_bias=v[1],
                            dpre_weight=v[2], dpre_bias=v[3], workspace=ws, **self.kinds())
        return out

    # -- the oracle's values and how far float32 may be from them --------------------------------------

    def check_fwd(self, out):
        x, h, gate = _np(self.x), _np(self.h), _np(self.gate)
        pw, pb, qw, qb = (_np(t) for t in self.vectors)
        y, u, ps, qs = T.residual_norm(x, h, gate, self.positions, self.post, self.pre, (pw, pb, qw, qb), self.skip,
                                       self.branch, self.eps)
        err = np.zeros_like(y)
        if h is not None:
            hat, _ = T.row_norm(h, self.post, None, None, self.eps)
            eh = _hat_error(h, hat, ps) if self.post != "none" else np.zeros_like(h)
            z = hat * _or(pw, 1) + _or(pb, 0)
            g = np.repeat(gate, self.positions, 0) if gate is not None else np.ones_like(z)
            ez = np.abs(_or(pw, 1)) * eh + 3 * U * (np.abs(z) + np.abs(_or(pb, 0)))
            err = np.abs(self.branch * g) * ez + 4 * U * (np.abs(self.skip * x) + np.abs(self.branch * g * z))
            _close(out["y"], y, err, self.stream, "y")
            if self.post != "none":
                _check_stats(out["post_stats"], ps, h, np.zeros((len(h), 1)))
        if self.pre != "none":
            hat, _ = T.row_norm(y, self.pre, None, None, self.eps)
            most = err.max(1, keepdims=True)
            eh = _hat_error(y, hat, qs) + qs[:, 1:] * most * (2 + np.abs(hat))
            eu = np.abs(_or(qw, 1)) * eh + 3 * U * (np.abs(u) + np.abs(_or(qb, 0)))
            _close(out["u"], u, eu, self.type, "u")
            _check_stats(out["pre_stats"], qs, y, most)

    def check_bwd(self, out):
        dy, du, y, h, gate = (_np(t) for t in (self.dy, self.du, self.y, self.h, self.gate))
        v = [_np(t) for t in self.vectors]
        ps, qs = _np(self.post_stats), _np(self.pre_stats)
        if ps is None:
            ps = np.tile([0.0, 1.0], (self.rows, 1))
        dx, dh, dgate, grads = T.residual_norm_backward(dy, du, y, h, gate, self.positions, self.post, self.pre, v, ps, qs,
                                                        self.skip, self.branch)
        over_rows = (self.rows / 256 + 21) * U
        t, et = _or(dy, np.zeros_like(dx)), np.zeros_like(dx)
        if self.pre != "none":
            xhat = (y - qs[:, :1]) * qs[:, 1:]
            dv = T.row_norm_backward(du, y, self.pre, qs, v[2])[0]
            et = _through_error(du * _or(v[2], 1), np.zeros_like(dx), xhat, qs[:, 1:]) + 2 * U * (np.abs(t) + np.abs(dv))
            t = t + dv
            for i, term in ((2, du * xhat), (3, du)):
                if out["vectors"][i] is not None:
                    _close(out["vectors"][i], grads[i], (over_rows + 4 * U) * np.abs(term).sum(0), "float32", f"pre {i}")
        _close(out["dx"], dx, np.abs(self.skip) * (et + U * np.abs(t)), self.stream, "dx")
        if h is None:
            return
        hat = (h - ps[:, :1]) * ps[:, 1:]
        z = hat * _or(v[0], 1) + _or(v[1], 0)
        g = np.repeat(gate, self.positions, 0) if gate is not None else np.ones_like(z)
        e = self.branch * t
        ee = np.abs(self.branch) * et + U * np.abs(e)
        if out["dgate"] is not None:
            each = ee * np.abs(z) + 6 * U * np.abs(e) * (np.abs(hat * _or(v[0], 1)) + np.abs(_or(v[1], 0)))
            fold = lambda a: a.reshape(-1, self.positions, self.c).sum(1)
            _close(out["dgate"], dgate, fold(each) + over_rows * fold(np.abs(e * z)), self.type, "dgate")
        dp, edp = e * g, np.abs(g) * ee + 2 * U * np.abs(e * g)
        for i, term, size in ((0, dp * hat, np.abs(hat)), (1, dp, np.ones_like(hat))):
            if out["vectors"][i] is not None:
                bound = (edp * size).sum(0) + (over_rows + 4 * U) * np.abs(term).sum(0)
                _close(out["vectors"][i], grads[i], bound, "float32", f"post {i}")
        q, eq = dp * _or(v[0], 1), np.abs(_or(v[0], 1)) * edp
        ed = _through_error(q, eq, hat, ps[:, 1:]) if self.post != "none" else eq + 2 * U * np.abs(q)
        _close(out["dh"], dh, ed, self.type, "dh")


def _or(a, other):
    return other if a is None else a


def _hat_error(v, hat, stats):
    mean, rstd = np.abs(stats[:, :1]), stats[:, 1:]
    return U * (K * rstd * np.abs(v).mean(1, keepdims=True) + 2 * rstd * (np.abs(v) + mean) + (K / 2 + 6) * np.abs(hat))


def _through_error(q, eq, hat, rstd):
    form = lambda a: np.abs(a) + np.abs(a).mean(1, keepdims=True) + np.abs(hat) * np.abs(a * hat).mean(1, keepdims=True)
    return rstd * ((K + 10) * U * form(q) + form(eq))


def _check_stats(got, ref, v, moved):
    """moved: how far the row's values may be off already."""
    got, size = _np(got), np.abs(v).mean(1)
    em = K * U * size + moved[:, 0]
    assert (np.abs(got[:, 0] - ref[:, 0]) <= em).all()
    # a mean that is off by em adds em^2 to the variance
    rel = (K / 2 + 6) * U + ref[:, 1] * moved[:, 0] + (ref[:, 1] * em) ** 2
    assert (np.abs(got[:, 1] - ref[:, 1]) <= rel * ref[:, 1]).all()


def _close(got, ref, err, dtype, what):
    got = _np(got)
    assert np.isfinite(got).all(), what
    bound = err + HALF[dtype] * (np.abs(ref) + err) + TINY[dtype] + 1e-37
    off = np.abs(got - ref) / bound
    assert off.max() <= 1, (what, float(off.max()))


def _variant(i, shape):
    """Norms, gate, vectors and types of case i, over all combinations in turn."""
    return dict(post=KINDS[i % 3], pre=KINDS[(i // 3 + 1) % 3], gate=i % 4 != 1, bias=i % 5 < 3, weight=i % 7 != 2)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=["x".join(map(str, s)) for s in SHAPES])
def test_both_directions(i, types):
    H.require_gpu()
    how = _variant(i + 2 * TYPES.index(types), SHAPES[i])
    H.note(f"residual norm {SHAPES[i]} {types} {how}")
    case = Case(SHAPES[i], types, **how)
    case.check_fwd(case.run_fwd())
    case.kept()
    case.check_bwd(case.run_bwd())


@pytest.mark.parametrize("pre", KINDS)
@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("gate", [False, True])
def test_every_pair_of_norms(post, pre, gate):
    H.require_gpu()
    H.note(f"residual norm {post} {pre} gate {gate}")
    for shape in ((66, 3, 72), (6, 3, 2048)):
        case = Case(shape, ("float32", "float32"), post, pre, gate=gate)
        case.check_fwd(case.run_fwd())
        case.kept()
        case.check_bwd(case.run_bwd())


@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_the_first_norm_of_a_stack_has_no_block(types, pre):
    H.require_gpu()
    H.note(f"residual norm without a block {types} {pre}")
    case = Case((37, 1, 264), types, "none", pre, block=False)
    case.check_fwd(case.run_fwd())
    case.kept()
    for dy in (True, False):
        case.dy = case.dy if dy else None
        case.check_bwd(case.run_bwd())


@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_skip_has_no_part_without_a_block(types, pre):
    """The forward's u is the norm of x itself, so its gradient is that of skip 1, which the oracle and differences
    of it confirm, bit for bit whatever skip and branch are."""
    import torch
    H.require_gpu()
    H.note(f"residual norm without a block, other skips {types} {pre}")
    case = Case((37, 1, 264), types, "none", pre, block=False)
    case.kept()
    fwd, bwd = case.run_fwd(), case.run_bwd()
    case.check_bwd(bwd)
    for skip, branch in ((0.5, 1.0), (0.0, 0.0), (-2.0, 3.0)):
        case.skip, case.branch = np.float32(skip), np.float32(branch)
        assert torch.equal(case.run_fwd()["u"], fwd["u"]), skip
        out = case.run_bwd()
        assert torch.equal(out["dx"], bwd["dx"]), skip
        assert all(torch.equal(a, b) for a, b in zip(out["vectors"][2:], bwd["vectors"][2:])), skip


def test_a_large_mean_keeps_the_variance():
    """A mean 100 times the deviation."""
    H.require_gpu()
    H.note("residual norm shifted rows")
    case = Case((200, 1, 128), ("float32", "float32"), "layer", "layer", shift=150.0)
    case.check_fwd(case.run_fwd())
    case.kept()
    case.check_bwd(case.run_bwd())


def test_without_a_gradient_from_elsewhere_and_with_few_gradients_asked_for():
    import torch
    H.require_gpu()
    H.note("residual norm: last block, and only dx and dh")
    case = Case((50, 5, 320), ("bfloat16", "bfloat16"), "rms", "layer", dy=False)
    case.kept()
    full = case.run_bwd()
    case.check_bwd(full)
    some = case.run_bwd(dgate=None, vectors=[None] * 4)
    assert torch.equal(some["dx"], full["dx"]) and torch.equal(some["dh"], full["dh"])
    one = case.run_bwd(vectors=[None, None, case.new("float32", 320), None])
    assert torch.equal(one["vectors"][2], full["vectors"][2]) and torch.equal(one["dgate"], full["dgate"])


@pytest.mark.parametrize("types", [TYPES[0], TYPES[1], TYPES[3]], ids="-".join)
def test_strided_rows_and_in_place(types):
    """Rows of wider buffers, whose other columns stay; y over x, u over h, dx over dy and y, dh over du."""
    import torch
    H.require_gpu()
    H.note(f"residual norm strided {types}")
    case = Case((45, 5, 104), types, "layer", "rms")
    plain = case.run_fwd()

    def wide(t, extra):
        buf = torch.full((t.shape[0], t.shape[1] + 2 * extra), 7.0, dtype=t.dtype, device="cuda")
        view = buf[:, extra:extra + t.shape[1]]
        view.copy_(t)
        return buf, view

    def untouched(buf, extra):
        return bool((buf[:, :extra] == 7).all()) and bool((buf[:, -extra:] == 7).all())
    bx, case.x = wide(case.x, 8)
    bh, case.h = wide(case.h, 16)
    bg, case.gate = wide(case.gate, 24)
    by, y = wide(plain["y"], 16)
    bu, u = wide(plain["u"], 8)
    y.fill_(0), u.fill_(0)
    out = case.run_fwd(y=y, u=u)
    assert torch.equal(y, plain["y"]) and torch.equal(u, plain["u"]) and untouched(by, 16) and untouched(bu, 8)
    assert torch.equal(out["post_stats"], plain["post_stats"]) and torch.equal(out["pre_stats"], plain["pre_stats"])
    case.kept()
    ref = case.run_bwd()
    bdx, dx = wide(ref["dx"], 8)
    bdh, dh = wide(ref["dh"], 8)
    bdg, dg = wide(ref["dgate"], 8)
    out = case.run_bwd(dx=dx, dh=dh, dgate=dg)
    assert untouched(bdx, 8) and untouched(bdh, 8) and untouched(bdg, 8)
    keep = case.dy.clone(), case.du.clone(), case.y.clone()
    over = case.run_bwd(dx=case.dy, dh=case.du)
    case.dy, case.du = keep[0], keep[1]
    over_y = case.run_bwd(dx=case.y)
    for o in (out, over, over_y):
        assert torch.equal(o["dx"], ref["dx"]) and torch.equal(o["dh"], ref["dh"]) and torch.equal(o["dgate"], ref["dgate"])
        assert all(torch.equal(a, b) for a, b in zip(o["vectors"], ref["vectors"]))
    case.run_fwd(y=case.x, u=case.h)
    assert torch.equal(case.x, plain["y"]) and torch.equal(case.h, plain["u"]) and untouched(bx, 8) and untouched(bh, 16)


def test_rows_without_values_and_without_finite_ones():
    """A zero row has deviation sqrt(eps); NaN and infinities stay in their row and, in a shared gate's gradient, its sample."""
    import torch
    H.require_gpu()
    H.note("residual norm special values")
    case = Case((30, 5, 136), ("float32", "float32"), "rms", "layer")
    case.x[3], case.h[3] = 0.0, 0.0
    case.check_fwd(case.run_fwd())
    clean = case.run_fwd()
    case.kept()
    grads = case.run_bwd()
    case.h[7, 11], case.x[12, 0], case.h[21, 5] = float("nan"), float("inf"), float("inf")
    bad = case.run_fwd()
    hit = [7, 12, 21]
    rest = [r for r in range(30) if r not in hit]
    for name in ("y", "u", "post_stats", "pre_stats"):
        assert torch.equal(bad[name][rest], clean[name][rest]), name
    assert torch.isnan(bad["y"][7]).all() and torch.isnan(bad["u"][hit]).all()
    assert torch.equal(bad["y"][12, 1:], clean["y"][12, 1:]) and torch.isinf(bad["y"][12, 0])
    case.h.copy_(torch.nan_to_num(case.h, nan=0.1, posinf=0.1))
    case.du[7, 11] = float("nan")
    bad = case.run_bwd()
    rest = [r for r in range(30) if r != 7]
    assert torch.isnan(bad["dx"][7]).all() and torch.isfinite(bad["dx"][rest]).all()
    assert torch.equal(bad["dx"][rest], grads["dx"][rest])
    samples = [s for s in range(6) if s != 1]
    assert torch.isnan(bad["dgate"][1]).all() and torch.isfinite(bad["dgate"][samples]).all()


def test_no_rows():
    import torch
    H.require_gpu()
    H.note("residual norm without rows")
    case = Case((0, 3, 64), ("bfloat16", "bfloat16"), "rms", "layer")
    case.run_fwd()
    case.y, case.post_stats, case.pre_stats = case.x, None, None
    out = case.run_bwd()
    assert all(bool((v == 0).all()) for v in out["vectors"])


def test_deterministic_on_another_stream_and_replayed():
    import torch
    H.require_gpu()
    H.note("residual norm streams and graphs")
    case = Case((5000, 50, 192), ("float32", "bfloat16"), "layer", "rms")
    case.kept()
    fwd, bwd = case.run_fwd(), case.run_bwd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd2, bwd2 = case.run_fwd(), case.run_bwd()
    torch.cuda.current_stream().wait_stream(side)
    flat = lambda f, b: [f["y"], f["u"], f["post_stats"], f["pre_stats"], b["dx"], b["dh"], b["dgate"]] + b["vectors"]
    assert all(torch.equal(a, b) for a, b in zip(flat(fwd, bwd), flat(fwd2, bwd2)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd3, bwd3 = case.run_fwd(), case.run_bwd()
    for turn in range(4):
        case.h.copy_(torch.randn(5000, 192, device="cuda") + turn)
        case.du.copy_(torch.randn(5000, 192, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in flat(fwd3, bwd3)]
        want = flat(case.run_fwd(), case.run_bwd())
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_offsets_beyond_32_bits():
    """Rows whose stride puts the last of them past 2^31 elements (and 2^32 bytes)."""
    import torch
    H.require_gpu()
    H.note("residual norm far rows")
    rows, c, ld = 2100, 64, 1 << 20
    case = Case((rows, 1, c), ("bfloat16", "bfloat16"), "rms", "layer")
    case.kept()
    fwd, bwd = case.run_fwd(), case.run_bwd()
    far = [torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)[:, :c] for _ in range(4)]
    far[0].copy_(case.x), far[1].copy_(case.h)
    case.x, case.h = far[0], far[1]
    out = case.run_fwd(y=far[2], u=far[3])
    assert torch.equal(far[2], fwd["y"]) and torch.equal(far[3], fwd["u"])
    far[0].copy_(case.y)
    case.y = far[0]
    out = case.run_bwd(dx=far[2], dh=far[3])
    assert torch.equal(far[2], bwd["dx"]) and torch.equal(far[3], bwd["dh"]) and torch.equal(out["dgate"], bwd["dgate"])
