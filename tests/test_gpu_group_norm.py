"""qha_group_norm_fwd and qha_group_norm_bwd against the float64 oracle.

Tolerances count roundings, u = 2^-24 the unit roundoff of float32, and one rounding of the output type
(half a step, eps / 2).  Forward: z = (x - mean) rstd w + b from float32 statistics (each off by u of
its value after float64 sums, or by about (4 + log2 of the row) u where a row is summed in float32)
costs at most 12 u (|x| + |mean|) rstd |w| + 2 u |b|; the activations have slopes below 1.13 and add
at most 8 u |z| of their own, so y is off by 1.13 of the first plus 16 u (|z| + 1).  Backward: dz carries
the slope's error, at most 1.2 of z's error plus 16 u, times |dy|; the group means average such
errors, and dx = rstd (q - mean q - xhat mean(q xhat)) adds 16 u of the sum of its terms' sizes.
Channel sums add at most (rows per partial + 32) u of the sum of their terms' sizes, in float32 runs
of at most 64 + rows / 1024 terms.
"""
import numpy as np
import pytest

import gpu_helpers as H
from oracle import train as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 0.0, "bfloat16": 0.0, "float16": 2.0 ** -25}      # half a step of subnormals
KINDS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}

# samples, positions, channels, groups
SHAPES = [(1, 1, 8, 1), (5, 1, 8, 8), (1001, 1, 128, 8), (300, 1, 256, 1), (77, 1, 40, 5), (33, 1, 1024, 32),
          (9, 1, 4096, 1), (5, 1, 2048, 64), (3, 1, 8192, 2), (7, 1, 1536, 3), (1, 1, 24, 24), (12, 1, 24, 4),
          (3, 97, 64, 8), (2, 1, 16, 2), (1, 3001, 128, 4), (17, 2, 40, 5), (2, 50, 2048, 16), (4, 9, 48, 12),
          (2, 33, 4096, 2), (40, 5, 256, 256), (2, 11, 1032, 3), (2, 3, 8192, 8192),
          (1, 3, 8192, 1)]


def _data(rows, c, dtype, seed, shift=0.25, scale=1.5):
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((rows, c)) * scale + shift).astype(np.float32)).to(getattr(torch, dtype))
    dy = torch.from_numpy(rng.standard_normal((rows, c)).astype(np.float32)).to(getattr(torch, dtype))
    w = (1 + 0.3 * rng.standard_normal(c)).astype(np.float32)
    b = (0.3 * rng.standard_normal(c)).astype(np.float32)
    return x, dy, w, b


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _wide(stat, positions, c, groups):
    """[samples, groups] statistics as [rows, c]."""
    return np.repeat(np.repeat(stat, c // groups, axis=1), positions, axis=0)


def _z_error(x, mean, rstd, w, b, positions, groups):
    c = x.shape[1]
    m, r = _wide(mean, positions, c, groups), _wide(rstd, positions, c, groups)
    return (12 + np.log2(c)) * U * (np.abs(x) + np.abs(m)) * r * np.abs(w) + 2 * U * np.abs(b)


def _run_fwd(x, w, b, groups, positions, kind, eps=1e-5, stats=True):
    import torch
    from quantized_halo_aggregation_amd import binding as B
    rows, c = x.shape
    n = rows // positions
    y = torch.full_like(x, float("nan"))
    mean, rstd = (torch.full((n, groups), float("nan"), device="cuda") for _ in range(2))
    ws = torch.empty(max(B.group_norm_workspace(rows, positions, c, groups), 16), dtype=torch.uint8, device="cuda")
    B.group_norm_fwd(x, y, groups, weight=w, bias=b, mean=mean if stats else None, rstd=rstd if stats else None, eps=eps,
                     act=KINDS[kind], positions=positions, workspace=ws)
    return y, mean, rstd


def _check_fwd(shape, dtype, kind, shift=0.25, affine=True, eps=1e-5):
    s, p, c, g = shape
    x, _, w, b = _data(s * p, c, dtype, 7, shift)
    y, mean, rstd = _run_fwd(x.cuda(), H.dev(w) if affine else None, H.dev(b) if affine else None, g, p, kind, eps)
    if not affine:
        w, b = np.ones(c), np.zeros(c)
    ref, rm, rr = T.group_norm(_np(x), w, b, g, p, eps, kind)
    size = np.abs(_np(x)).reshape(-1, p, g, c // g).max((1, 3))
    assert (np.abs(H.host(mean) - rm) <= (2 + np.log2(c)) * U * size).all()
    # the deviations carry the mean's error, which is a share size * rstd of them
    assert (np.abs(H.host(rstd) - rr) <= ((8 + np.log2(c)) * U * (1 + ((2 + np.log2(c)) * U * size * rr) * size * rr)) * rr).all()
    z = np.abs(T.group_norm(_np(x), w, b, g, p, eps, "none")[0])
    bound = 1.13 * _z_error(_np(x), rm, rr, w, b, p, g) + 16 * U * (z + 1)
    bound = bound + HALF[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    err = np.abs(_np(y) - ref)
    assert np.isfinite(_np(y)).all()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dtype):
    H.require_gpu()
    kind = list(KINDS)[(shape[2] // 8 + shape[3]) % 4]
    H.note(f"group norm fwd {shape} {dtype} {kind}")
    _check_fwd(shape, dtype, kind)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", [(65, 1, 128, 4), (2, 130, 64, 2)], ids=["rows", "maps"])
def test_forward_without_affine_and_with_a_large_mean(shape, kind):
    """A mean 100 times the deviation: the statistics must not lose the variance."""
    H.require_gpu()
    H.note(f"group norm fwd {shape} {kind} plain and shifted")
    _check_fwd(shape, "float32", kind, affine=False)
    _check_fwd(shape, "float32", kind, shift=150.0)


def _check_bwd(shape, dtype, kind, affine=True, strided=False):
    import torch
    from quantized_halo_aggregation_amd import binding as B
    s, p, c, g = shape
    rows = s * p
    x, dy, w, b = _data(rows, c, dtype, 11)
    if not affine:
        w, b = np.ones(c, np.float32), np.zeros(c, np.float32)
    _, mean, rstd = T.group_norm(_np(x), w, b, g, p, 1e-5, kind)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    xd, dyd = x.cuda(), dy.cuda()
    dx = torch.full_like(xd, float("nan"))
    dw, db = (torch.full((c,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.empty(max(B.group_norm_workspace(rows, p, c, g, backward=True), 16), dtype=torch.uint8, device="cuda")

    def call():
        B.group_norm_bwd(dyd, xd, H.dev(mean), H.dev(rstd), dx, g, weight=H.dev(w) if affine else None,
                         bias=H.dev(b) if affine else None, dweight=dw, dbias=db, act=KINDS[kind], positions=p,
                         workspace=ws)
    call()
    rdx, rdw, rdb = T.group_norm_backward(_np(dy), _np(x), mean, rstd, w, b, g, p, kind)
    m, r = _wide(mean.astype(np.float64), p, c, g), _wide(rstd.astype(np.float64), p, c, g)
    xhat = (_np(x) - m) * r
    slope = np.abs(T.act_slope(xhat * w + b, kind))
    zerr = _z_error(_np(x), mean.astype(np.float64), rstd.astype(np.float64), w, b, p, g)
    dz = np.abs(_np(dy)) * slope
    edz = np.abs(_np(dy)) * ((0 if kind in ("none", "relu") else 1.2 * zerr + 16 * U) + 2 * U * slope)
    exh = 4 * U * (np.abs(_np(x)) + np.abs(m)) * r
    grp = lambda t: _wide(t.reshape(s, p, g, -1).mean((1, 3)), p, c, g)
    aw = np.abs(w)
    terms = aw * dz + grp(aw * dz) + np.abs(xhat) * grp(aw * dz * np.abs(xhat))
    run = 64 + rows / 1024 + 32
    bound = r * (aw * edz + grp(aw * edz) + exh * grp(aw * dz * np.abs(xhat)) +
                 np.abs(xhat) * grp(aw * (edz * np.abs(xhat) + dz * exh)) + run * U * terms)
    bound = bound + HALF[dtype] * (np.abs(rdx) + bound) + TINY[dtype]
    err = np.abs(_np(dx) - rdx)
    assert (err <= bound).all(), float((err / bound).max())
    for got, ref, size, e in ((dw, rdw, dz * np.abs(xhat), edz * np.abs(xhat) + dz * exh), (db, rdb, dz, edz)):
        bnd = e.sum(0) + run * U * size.sum(0)
        assert (np.abs(H.host(got) - ref) <= bnd).all(), float((np.abs(H.host(got) - ref) / bnd).max())
    first = [t.clone() for t in (dx, dw, db)]
    call()
    for a, t in zip(first, (dx, dw, db)):
        assert torch.equal(a, t), "results must be deterministic"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, dtype):
    H.require_gpu()
    kind = list(KINDS)[(shape[2] // 8 + shape[3]) % 4]
    H.note(f"group norm bwd {shape} {dtype} {kind}")
    _check_bwd(shape, dtype, kind)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", [(20011, 1, 32, 2), (3, 4001, 16, 1)], ids=["rows", "maps"])
def test_backward_of_many_rows(shape, kind):
    H.require_gpu()
    H.note(f"group norm bwd {shape} {kind}")
    _check_bwd(shape, "float32", kind, affine=kind != "silu")


SMALL = [(700, 4, 32, 1), (501, 9, 8, 1), (333, 2, 128, 4), (77, 7, 40, 5), (65, 3, 1032, 3), (50, 6, 256, 32), (9, 25, 320, 8),
         (5, 2, 4096, 4), (40, 31, 16, 2), (3, 1000, 8, 1), (6, 3, 2048, 1), (19, 16, 64, 4),
         (260, 2, 4096, 4), (257, 97, 64, 8), (300, 3, 2048, 1)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", SMALL, ids=lambda s: "x".join(map(str, s)))
def test_small_samples(shape, dtype):
    """Samples that a team of threads holds whole: every team size and way of summing groups, and one just over."""
    H.require_gpu()
    kind = list(KINDS)[(shape[1] + shape[3]) % 4]
    H.note(f"group norm small {shape} {dtype} {kind}")
    _check_fwd(shape, dtype, kind)
    _check_bwd(shape, dtype, kind)


def test_strided_rows_and_in_place():
    """Column slices of wider buffers (the layout of concatenated halves), y in x's place, dx in dy's."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    for rows, p, c, g in ((301, 1, 64, 4), (300, 100, 64, 4)):
        H.note(f"group norm strided rows={rows} positions={p}")
        x, dy, w, b = _data(rows, c, "float32", 5)
        y, mean, rstd = _run_fwd(x.cuda(), H.dev(w), H.dev(b), g, p, "silu")
        wide = torch.full((rows, 3 * c), 7.0, device="cuda")
        wide[:, c:2 * c] = x.cuda()
        part = wide[:, c:2 * c]
        ws = torch.empty(max(B.group_norm_workspace(rows, p, c, g, True), 16), dtype=torch.uint8, device="cuda")
        B.group_norm_fwd(part, part, g, weight=H.dev(w), bias=H.dev(b), act=B.ACT_SILU, positions=p, workspace=ws)
        assert torch.equal(part, y)
        assert (wide[:, :c] == 7).all() and (wide[:, 2 * c:] == 7).all()
        dx = torch.empty_like(x, device="cuda")
        args = dict(weight=H.dev(w), bias=H.dev(b), act=B.ACT_SILU, positions=p, workspace=ws)
        B.group_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, dx, g, **args)
        wide[:, c:2 * c] = dy.cuda()
        B.group_norm_bwd(part, x.cuda(), mean, rstd, part, g, **args)
        assert torch.equal(part, dx)


def test_rows_without_spread_and_values_that_are_not_finite():
    """A constant group has variance 0: y = act(b) and finite gradients.  NaN and infinity stay in their
    own sample's group."""
    H.require_gpu()
    import torch
    for p in (1, 6):
        H.note(f"group norm degenerate positions={p}")
        x = torch.randn(4 * p, 32, generator=torch.Generator().manual_seed(1))
        x[:p, :16] = 3.0
        x[p, 20] = float("nan")
        x[3 * p, 1] = float("inf")
        w, b = torch.full((32,), 2.0), torch.linspace(-1, 1, 32)
        y, mean, rstd = _run_fwd(x.cuda(), w.cuda(), b.cuda(), 2, p, "none")
        got = _np(y)
        assert np.array_equal(got[:p, :16], np.broadcast_to(b.numpy()[:16], (p, 16)).astype(np.float64))
        bad = np.zeros((4 * p, 32), bool)
        bad[p:2 * p, 16:] = True
        bad[3 * p:, :16] = True
        assert np.isfinite(got[~bad]).all() and np.isnan(got[p:2 * p, 16:]).all() and not np.isfinite(got[3 * p:, :16]).any()
        ref = T.group_norm(np.where(np.isfinite(x.numpy()), x.numpy(), 0), w.numpy(), b.numpy(), 2, p, 1e-5, "none")[0]
        keep = ~bad
        keep[:p, :16] = False
        assert np.abs(got - ref)[keep].max() < 1e-4


def test_no_rows():
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.note("group norm without rows")
    x = torch.empty(0, 16, device="cuda")
    st = torch.empty(0, 2, device="cuda")
    dw, db = torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    B.group_norm_fwd(x, x, 2)
    B.group_norm_bwd(x, x, st, st, x, 2, dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_graph_replays_equal_the_eager_call():
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    for rows, p in ((500, 1), (600, 200)):
        H.note(f"group norm graph positions={p}")
        x, dy, w, b = (t.cuda() if torch.is_tensor(t) else H.dev(t) for t in _data(rows, 64, "bfloat16", 9))
        n = rows // p
        ws = torch.empty(max(B.group_norm_workspace(rows, p, 64, 4, True), B.group_norm_workspace(rows, p, 64, 4), 16),
                         dtype=torch.uint8, device="cuda")
        out = [torch.zeros_like(x), torch.zeros_like(x), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda"),
               torch.zeros(n, 4, device="cuda"), torch.zeros(n, 4, device="cuda")]

        def step():
            y, dx, dw, db, mean, rstd = out
            B.group_norm_fwd(x, y, 4, weight=w, bias=b, mean=mean, rstd=rstd, act=B.ACT_GELU, positions=p, workspace=ws)
            B.group_norm_bwd(dy, x, mean, rstd, dx, 4, weight=w, bias=b, dweight=dw, dbias=db, act=B.ACT_GELU,
                             positions=p, workspace=ws)
        step()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step()
        for k in range(4):
            x.add_(0.125 * k)
            dy.mul_(1.5)
            step()
            want = [t.clone() for t in out]
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, t in zip(want, out):
                assert torch.equal(a, t), k


@pytest.mark.parametrize("shape", [(700, 1, 4, 1), (33, 1, 4, 2), (50, 1, 4, 4), (3, 1000, 4, 1), (2, 3001, 4, 2), (5, 60, 4, 1),
                                   (301, 1, 12, 3), (40, 1, 12, 2), (3, 500, 12, 3), (2, 1500, 12, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_four_and_twelve_float32_channels(shape):
    """Widths that only float32 has: one or three vectors a row, groups of whole vectors and groups that cut them."""
    H.require_gpu()
    for kind in ("relu", "silu"):
        H.note(f"group norm narrow {shape} {kind}")
        _check_fwd(shape, "float32", kind)
        _check_bwd(shape, "float32", kind)


@pytest.mark.parametrize("kind", list(KINDS))
def test_every_activation_keeps_nan(kind):
    """A NaN in x reaches every y and dx of its sample's group, whatever the activation, in rows, small and large samples,
    and no other; a NaN weight or bias reaches its channel."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    for s, p, c in ((6, 1, 32), (4, 6, 32), (3, 400, 32), (4, 1, 12), (3, 700, 12)):
        H.note(f"group norm NaN {kind} {s}x{p}x{c}")
        x, dy, w, b = _data(s * p, c, "float32", 3)
        x[p, c // 2 + 1] = float("nan")
        b[0] = float("nan")
        y, mean, rstd = _run_fwd(x.cuda(), H.dev(w), H.dev(b), 2, p, kind)
        bad = np.zeros((s * p, c), bool)
        bad[p:2 * p, c // 2:] = True
        hit = bad.copy()
        hit[:, 0] = True
        assert np.array_equal(np.isnan(_np(y)), hit)
        dx = torch.zeros(s * p, c, device="cuda")
        ws = torch.empty(max(B.group_norm_workspace(s * p, p, c, 2, True), 16), dtype=torch.uint8, device="cuda")
        b[0] = 0.0
        B.group_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, dx, 2, weight=H.dev(w), bias=H.dev(b), act=KINDS[kind],
                         positions=p, workspace=ws)
        assert np.array_equal(np.isnan(_np(dx)), bad)
