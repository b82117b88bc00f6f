"""qha_gated_project and qha_gated_backward against the float64 oracle.

Tolerances count roundings, u = 2^-24 the unit roundoff of float32.  A dot product of length L sums
exact products (16-bit types) or part products that total the product to 2^-23 (float32) in float32
accumulators, whose additions may truncate: at most 2 (L + 8) u of the sum of its terms' sizes S.
H = act(G) U is off by 1.13 |U| eG + |act(G)| eU (slopes are below 1.13) and 16 u of (|G| + 1) |U|; stored
values are rounded once more, by at most half a step (eps / 2).  dG = dH U act'(G) and dU = dH act(G) come
from the stored G and U: 16 u of |dH U| (1 + |G|) and of |dH| (1 + |G|); as 16-bit operands they are
rounded by half a step.  Those errors go through dA and dW with the sizes of the other factor.
"""
import numpy as np
import pytest

import gpu_helpers as H
from oracle import train as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 1e-44, "bfloat16": 1e-40, "float16": 2.0 ** -25}      # half a step of subnormals
KINDS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
SHAPES = [(1, 8, 8), (1, 512, 256), (2, 64, 1024), (7, 40, 24), (16, 128, 136), (17, 8, 512), (33, 200, 64), (64, 72, 200),
          (100, 256, 128), (129, 136, 128), (300, 64, 264), (513, 328, 72), (1001, 128, 128), (2500, 16, 16),
          (1030, 512, 320)]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _data(m, n, k, dtype, seed):
    import torch
    rng = np.random.default_rng(seed)
    mk = lambda *s, f=1.0: torch.from_numpy((rng.standard_normal(s) * f).astype(np.float32)).to(getattr(torch, dtype))
    return mk(m, k), mk(n, k, f=1 / np.sqrt(k)), mk(n, k, f=1 / np.sqrt(k)), mk(m, n)


def _space(need):
    import torch
    return torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


def _forward(a, wg, wu, kind, kept=True):
    import torch
    from quantized_halo_aggregation_amd import binding as B
    m, n, k = a.shape[0], wg.shape[0], a.shape[1]
    out = [torch.full((m, n), float("nan"), dtype=a.dtype, device="cuda") for _ in range(3)]
    B.gated_project(a, wg, wu, out[0], gate=out[1] if kept else None, up=out[2] if kept else None, act=KINDS[kind],
                    workspace=_space(B.gated_project_workspace(a.dtype, m, n, k)))
    return out


def _check_forward(m, n, k, dtype, kind):
    a, wg, wu, _ = _data(m, n, k, dtype, m + n + k)
    h, gate, up = _forward(a.cuda(), wg.cuda(), wu.cuda(), kind)
    rh, rg, ru = T.gated(_np(a), _np(wg), _np(wu), kind)
    eg, eu = (2 * (k + 8) * U * (np.abs(_np(a)) @ np.abs(_np(w)).T) for w in (wg, wu))
    fin = lambda e, ref: e + HALF[dtype] * (np.abs(ref) + e) + TINY[dtype]
    eh = 1.13 * (np.abs(ru) + eu) * eg + np.abs(T.act(rg, kind)) * eu + 16 * U * (np.abs(rg) + 1) * np.abs(ru)
    for name, got, ref, e in (("gate", gate, rg, eg), ("up", up, ru, eu), ("h", h, rh, eh)):
        err, bound = np.abs(_np(got) - ref), fin(e, ref)
        assert (err <= bound).all(), (name, float((err / bound).max()))
    alone, _, _ = _forward(a.cuda(), wg.cuda(), wu.cuda(), kind, kept=False)
    assert (alone == h).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dtype):
    H.require_gpu()
    kind = list(KINDS)[sum(shape) // 8 % 4]
    H.note(f"gated fwd {shape} {dtype} {kind}")
    _check_forward(*shape, dtype, kind)


@pytest.mark.parametrize("shape", [(5, 12, 20), (200, 68, 36), (131, 4, 4)], ids=lambda s: "x".join(map(str, s)))
def test_float32_widths_that_are_multiples_of_four(shape):
    H.require_gpu()
    H.note(f"gated fwd and bwd {shape} float32")
    _check_forward(*shape, "float32", "silu")
    _check_backward(*shape, "float32", "silu")


def _check_backward(m, n, k, dtype, kind):
    import torch
    from quantized_halo_aggregation_amd import binding as B
    a, wg, wu, dh = _data(m, n, k, dtype, m + 3 * n + k)
    gate = (_np(a) @ _np(wg).T)
    up = (_np(a) @ _np(wu).T)
    t = getattr(torch, dtype)
    gate, up = (torch.from_numpy(x.astype(np.float32)).to(t) for x in (gate, up))
    da = torch.full((m, k), float("nan"), dtype=t, device="cuda")
    dwg, dwu = (torch.full((n, k), float("nan"), device="cuda") for _ in range(2))
    args = [x.cuda() for x in (dh, gate, up, a, wg, wu)]
    ws = _space(B.gated_backward_workspace(t, m, n, k))
    B.gated_backward(*args, da, dwg, dwu, act=KINDS[kind], workspace=ws)
    fdh, fg, fu, fa, fwg, fwu = (_np(x) for x in (dh, gate, up, a, wg, wu))
    rda, rdwg, rdwu = T.gated_backward(fdh, fg, fu, fa, fwg, fwu, kind)
    dg, du = np.abs(fdh * fu * T.act_slope(fg, kind)), np.abs(fdh * T.act(fg, kind))
    half = 0.0 if dtype == "float32" else HALF[dtype]
    tiny = 0.0 if dtype == "float32" else TINY[dtype]
    edg = 16 * U * np.abs(fdh * fu) * (1 + np.abs(fg)) + half * dg + tiny
    edu = 16 * U * np.abs(fdh) * (1 + np.abs(fg)) + half * du + tiny
    dg, du = dg + edg, du + edu
    awg, awu, aa = np.abs(fwg), np.abs(fwu), np.abs(fa)
    eda = edg @ awg + edu @ awu + 2 * (2 * n + 8) * U * (dg @ awg + du @ awu)
    eda = eda + HALF[dtype] * (np.abs(rda) + eda) + TINY[dtype]
    for name, got, ref, e in (("da", da, rda, eda), ("dwg", dwg, rdwg, edg.T @ aa + 2 * (m + 8) * U * (dg.T @ aa)),
                              ("dwu", dwu, rdwu, edu.T @ aa + 2 * (m + 8) * U * (du.T @ aa))):
        err = np.abs(_np(got) - ref)
        assert (err <= e + 1e-44).all(), (name, float((err / (e + 1e-44)).max()))
    again = [torch.empty_like(x) for x in (dwg, dwu)]
    B.gated_backward(*args, None, *again, act=KINDS[kind], workspace=ws)       # a first layer needs no dA
    assert torch.equal(again[0], dwg) and torch.equal(again[1], dwu), "results must be deterministic"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, dtype):
    H.require_gpu()
    kind = list(KINDS)[(sum(shape) // 8 + 1) % 4]
    H.note(f"gated bwd {shape} {dtype} {kind}")
    _check_backward(*shape, dtype, kind)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_many_rows(dtype):
    H.require_gpu()
    H.note(f"gated 20011 rows {dtype}")
    _check_forward(20011, 128, 128, dtype, "silu")
    _check_backward(20011, 128, 64, dtype, "relu")


@pytest.mark.parametrize("shape,dtype", [((8200, 2056, 72), "bfloat16"), ((8200, 2056, 72), "float16"),
                                         ((33000, 136, 40), "float32"), ((66000, 8, 24), "float32"),
                                         ((17000, 264, 136), "bfloat16"), ((17000, 136, 260), "float32")],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_large_tiles(shape, dtype):
    """Enough tiles for the wider tile shapes, each with ragged last rows, columns and steps."""
    H.require_gpu()
    H.note(f"gated large tiles {shape} {dtype}")
    if shape[1] % 8 == 0 or dtype == "float32":
        _check_forward(*shape, dtype, "silu")
        _check_backward(*shape, dtype, "silu")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", [(1, 72, 4104), (15, 1000, 520), (32, 24, 264), (48, 520, 1032), (65, 136, 512), (128, 2048, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_few_rows(shape, dtype):
    """The kernel for few rows over its row counts, with reductions longer and shorter than a block's turn, and
    split gradients."""
    H.require_gpu()
    H.note(f"gated few rows {shape} {dtype}")
    _check_forward(*shape, dtype, "silu")
    _check_backward(*shape, dtype, "gelu")


@pytest.mark.parametrize("dtype", ["float32", "float16"])
def test_strided_operands(dtype):
    """Every array a column slice of a wider buffer: the same bits, and nothing written beside them."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    t = getattr(torch, dtype)
    for m, n, k in ((3, 64, 72), (300, 136, 72)):
        H.note(f"gated strided {m} {dtype}")
        a, wg, wu, dh = (x.cuda() for x in _data(m, n, k, dtype, 4))
        h, gate, up = _forward(a, wg, wu, "gelu")
        da = torch.empty_like(a)
        dws = [torch.empty(n, k, device="cuda") for _ in range(2)]
        ws = _space(B.gated_backward_workspace(t, m, n, k))
        B.gated_backward(dh, gate, up, a, wg, wu, da, *dws, act=3, workspace=ws)
        wide = []

        def slot(x, fill=True):
            buf = torch.full((x.shape[0], x.shape[1] + 32), 5.0, dtype=x.dtype, device="cuda")
            view = buf[:, 16:16 + x.shape[1]]
            if fill:
                view.copy_(x)
            wide.append((buf, x.shape[1]))
            return view
        sa, sg, su, sdh = (slot(x) for x in (a, wg, wu, dh))
        oh, og, ou = (slot(h, False) for _ in range(3))
        B.gated_project(sa, sg, su, oh, gate=og, up=ou, act=3, workspace=_space(B.gated_project_workspace(t, m, n, k)))
        assert torch.equal(oh, h) and torch.equal(og, gate) and torch.equal(ou, up)
        oda, odg, odu = slot(da, False), slot(dws[0], False), slot(dws[1], False)
        B.gated_backward(sdh, og, ou, sa, sg, su, oda, odg, odu, act=3, workspace=ws)
        assert torch.equal(oda, da) and torch.equal(odg, dws[0]) and torch.equal(odu, dws[1])
        for buf, w in wide:
            assert (buf[:, :16] == 5).all() and (buf[:, 16 + w:] == 5).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_every_array_with_a_stride_of_its_own(dtype):
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    t = getattr(torch, dtype)
    for m, n, k in ((2, 72, 64), (200, 136, 200)):
        H.note(f"gated own strides {m} {dtype}")
        a, wg, wu, dh = (x.cuda() for x in _data(m, n, k, dtype, 6))
        h, gate, up = _forward(a, wg, wu, "silu")
        da, dws = torch.empty_like(a), [torch.empty(n, k, device="cuda") for _ in range(2)]
        ws = _space(B.gated_backward_workspace(t, m, n, k))
        B.gated_backward(dh, gate, up, a, wg, wu, da, *dws, workspace=ws)
        pad = iter(range(8, 200, 8))

        def own(x):
            view = torch.full((x.shape[0], x.shape[1] + next(pad)), 3.0, dtype=x.dtype, device="cuda")[:, :x.shape[1]]
            return view.copy_(x)
        sa, sg, su, sdh, oh, og, ou, oda, odg, odu = (own(x) for x in (a, wg, wu, dh, h * 0, gate * 0, up * 0, da * 0, dws[0] * 0, dws[1] * 0))
        B.gated_project(sa, sg, su, oh, gate=og, up=ou, workspace=_space(B.gated_project_workspace(t, m, n, k)))
        assert torch.equal(oh, h) and torch.equal(og, gate) and torch.equal(ou, up)
        B.gated_backward(sdh, og, ou, sa, sg, su, oda, odg, odu, workspace=ws)
        assert torch.equal(oda, da) and torch.equal(odg, dws[0]) and torch.equal(odu, dws[1])


def test_values_that_are_not_finite_stay_in_their_rows():
    H.require_gpu()
    import torch
    for m in (5, 200):
        for dtype in ("float32", "bfloat16"):
            H.note(f"gated not finite {m} {dtype}")
            a, wg, wu, _ = _data(m, 64, 40, dtype, 8)
            a[m - 1, 3], a[1, 0] = float("nan"), float("inf")
            h, _, _ = _forward(a.cuda(), wg.cuda(), wu.cuda(), "silu")
            bad = ~np.isfinite(_np(h)).all(1)
            assert bad[m - 1] and set(np.flatnonzero(bad)) <= {1, m - 1}


def test_no_rows():
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.note("gated without rows")
    for t in (torch.float32, torch.bfloat16):
        a, h = torch.empty(0, 16, dtype=t, device="cuda"), torch.empty(0, 24, dtype=t, device="cuda")
        w = torch.ones(24, 16, dtype=t, device="cuda")
        dws = [torch.ones(24, 16, device="cuda") for _ in range(2)]
        B.gated_project(a, w, w, h)
        B.gated_backward(h, h, h, a, w, w, a, *dws, workspace=_space(B.gated_backward_workspace(t, 0, 24, 16)))
        assert all((d == 0).all() for d in dws)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_graph_replays_equal_the_eager_call(dtype):
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    t = getattr(torch, dtype)
    for m, n, k in ((4, 64, 128), (700, 136, 64)):
        H.note(f"gated graph {m} {dtype}")
        a, wg, wu, dh = (x.cuda() for x in _data(m, n, k, dtype, 2))
        out = [torch.zeros(m, n, dtype=t, device="cuda") for _ in range(3)] + [torch.zeros_like(a)] + \
              [torch.zeros(n, k, device="cuda") for _ in range(2)]
        ws = _space(max(B.gated_backward_workspace(t, m, n, k), B.gated_project_workspace(t, m, n, k)))

        def step():
            B.gated_project(a, wg, wu, out[0], gate=out[1], up=out[2], workspace=ws)
            B.gated_backward(dh, out[1], out[2], a, wg, wu, *out[3:], workspace=ws)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(4):
            a.mul_(1.25)
            wg.add_(0.0625 * i)
            step()
            want = [x.clone() for x in out]
            for x in out:
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(want, out):
                assert torch.equal(x, y), i


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kind", list(KINDS))
def test_every_activation_keeps_nan(kind, dtype):
    """A row of A with a NaN has NaN in all of H, and a NaN among the kept gates makes that row's dA NaN, whatever the
    activation; other rows are as without it."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    for m in (5, 200):
        H.note(f"gated NaN {kind} {dtype} {m}")
        a, wg, wu, dh = _data(m, 64, 40, dtype, 8)
        clean = [t.clone() for t in _forward(a.cuda(), wg.cuda(), wu.cuda(), kind)]
        a[m - 2, 3] = float("nan")
        h, _, _ = _forward(a.cuda(), wg.cuda(), wu.cuda(), kind)
        rows = np.arange(m) != m - 2
        assert np.isnan(_np(h)[m - 2]).all() and np.array_equal(_np(h)[rows], _np(clean[0])[rows])
        h, gate, up = clean
        ws = _space(B.gated_backward_workspace(a.dtype, m, 64, 40))
        da = [torch.zeros(m, 40, dtype=a.dtype, device="cuda") for _ in range(2)]
        dws = [torch.zeros(64, 40, device="cuda") for _ in range(2)]
        a[m - 2, 3] = 0.5
        for out in da:
            B.gated_backward(dh.cuda(), gate, up, a.cuda(), wg.cuda(), wu.cuda(), out, *dws, act=KINDS[kind], workspace=ws)
            gate[m - 2, 5] = float("nan")
        assert np.isfinite(_np(da[0])).all() and np.isnan(_np(da[1])[m - 2]).all()
        assert np.array_equal(_np(da[1])[rows], _np(da[0])[rows])
        # the gate's column is NaN in dup, and in dgate where the slope needs the gate
        assert np.isnan(_np(dws[1])[5]).all() and np.isfinite(np.delete(_np(dws[1]), 5, 0)).all()


def _check_f16_range(m, n, k, kind, rows, cols, weights):
    """f16 gradients whose dH has the sizes `rows` and whose up has the sizes `cols` (cycled).

    A term of [dG dU] carries 16 u of |dH U| (1 + |G|) or |dH| (1 + |G|) as above.  For dW it enters in two parts, scaled so that its
    column's largest is in [2^14, 2^15): 2^-22 of itself, or half of f16's last step 2^-24 against 2^14 at least, 2^-39 of
    that largest.  For dA in one, scaled by its row: 2^-11 of itself or 2^-39 of the row's largest."""
    import torch
    from quantized_halo_aggregation_amd import binding as B
    rng = np.random.default_rng(m + n + k)
    half = lambda x: torch.from_numpy(np.asarray(x, np.float32)).to(torch.float16)
    fill = lambda sizes, count: np.resize(np.asarray(sizes, np.float64), count)
    a, gate = half(rng.standard_normal((m, k))), half(rng.standard_normal((m, n)))
    dh = half(rng.standard_normal((m, n)) * fill(rows, m)[:, None])
    up = half(rng.standard_normal((m, n)) * fill(cols, n))
    wg, wu = (half(rng.standard_normal((n, k)) * weights) for _ in range(2))
    da = torch.full((m, k), float("nan"), dtype=torch.float16, device="cuda")
    dw = [torch.full((n, k), float("nan"), device="cuda") for _ in range(2)]
    B.gated_backward(*(x.cuda() for x in (dh, gate, up, a, wg, wu)), da, *dw, act=KINDS[kind],
                     workspace=_space(B.gated_backward_workspace(torch.float16, m, n, k)))
    fdh, fg, fu, fa, fwg, fwu = (_np(x) for x in (dh, gate, up, a, wg, wu))
    rda, *rdw = T.gated_backward(fdh, fg, fu, fa, fwg, fwu, kind)
    aa, aw = np.abs(fa), (np.abs(fwg), np.abs(fwu))
    terms = np.abs(fdh * fu * T.act_slope(fg, kind)), np.abs(fdh * T.act(fg, kind))
    own = 16 * U * np.abs(fdh * fu) * (1 + np.abs(fg)), 16 * U * np.abs(fdh) * (1 + np.abs(fg))
    for name, got, ref, t, e in zip(("dwg", "dwu"), dw, rdw, terms, own):
        e = e + 2.0 ** -22 * t + 2.0 ** -39 * t.max(0)
        bound = e.T @ aa + 2 * (m + 8) * U * ((t + e).T @ aa)
        err = np.abs(_np(got) - ref)
        assert (err <= bound).all(), (name, float((err / bound).max()))
    top = np.maximum(terms[0].max(1), terms[1].max(1))[:, None]
    e = sum((o + 2.0 ** -11 * t + 2.0 ** -39 * top) @ w + 2 * (2 * n + 8) * U * (t @ w) for o, t, w in zip(own, terms, aw))
    e = e + HALF["float16"] * (np.abs(rda) + e) + TINY["float16"]
    fits = np.abs(rda) + e < 65504
    err = np.abs(_np(da) - rda)
    assert fits.mean() > 0.9 and (err <= e)[fits].all(), ("da", float((err / e)[fits].max()))


@pytest.mark.parametrize("rows,cols,weights", [((1e-5,), (1.0,), 0.1), ((1e-3,), (1e-4,), 0.1), ((3e2,), (1e4,), 1e-4),
                                               ((1e-6, 1.0, 1e4), (1e-4, 1.0, 1e3, 1e-2), 1e-4), ((1e4, 1e-7), (1.0,), 0.05)],
                         ids=["small", "product_underflows", "product_overflows", "mixed", "rows_far_apart"])
@pytest.mark.parametrize("shape", [(1, 8, 16), (33, 72, 40), (300, 520, 264), (2500, 64, 128), (700, 1032, 72)],
                         ids=lambda s: "x".join(map(str, s)))
def test_f16_gradients_of_any_size(shape, rows, cols, weights):
    """dgate and dup leave f16's range in both directions; the weight gradients are float32 and stay exact to their terms."""
    H.require_gpu()
    kind = ["silu", "none", "gelu", "relu"][sum(shape) // 8 % 4]
    H.note(f"gated f16 range {shape} {rows} {cols} {kind}")
    _check_f16_range(*shape, kind, rows, cols, weights)


def test_f16_gradients_that_are_not_finite():
    """An infinite dH makes its columns' weight gradients infinite with A's signs and its row of dA not finite; all else is as
    without it."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    m, n, k = 150, 72, 40
    H.note("gated f16 infinite gradient")
    a, wg, wu, dh = _data(m, n, k, "float16", 5)
    a[7] = torch.where(a[7] == 0, torch.ones_like(a[7]), a[7])
    gate, up = torch.full((m, n), 2.0, dtype=torch.float16), torch.full((m, n), 3.0, dtype=torch.float16)
    ws = _space(B.gated_backward_workspace(torch.float16, m, n, k))
    runs = []
    for value in (0.0, float("inf")):
        dh[7, 11] = value
        out = [torch.zeros(m, k, dtype=torch.float16, device="cuda")] + [torch.zeros(n, k, device="cuda") for _ in range(2)]
        B.gated_backward(*(x.cuda() for x in (dh, gate, up, a, wg, wu)), *out, act=0, workspace=ws)
        runs.append([_np(x) for x in out])
    for i, hit in ((0, 7), (1, 11), (2, 11)):
        keep = np.arange(runs[0][i].shape[0]) != hit
        assert np.array_equal(runs[0][i][keep], runs[1][i][keep])
    assert not np.isfinite(runs[1][0][7]).any()
    assert (runs[1][1][11] == np.inf * np.sign(_np(a)[7])).all() and (runs[1][2][11] == runs[1][1][11]).all()


def test_f16_gradients_in_a_graph():
    """The sizes are found again in every replay."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    m, n, k = 700, 136, 64
    H.note("gated f16 graph")
    a, wg, wu, dh = (x.cuda() for x in _data(m, n, k, "float16", 2))
    _, gate, up = _forward(a, wg, wu, "silu")
    out = [torch.zeros_like(a)] + [torch.zeros(n, k, device="cuda") for _ in range(2)]
    ws = _space(B.gated_backward_workspace(torch.float16, m, n, k))
    step = lambda: B.gated_backward(dh, gate, up, a, wg, wu, *out, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for scale in (1e-3, 1e-2, 1e4, 1e-4):
        dh.mul_(scale)
        step()
        want = [x.clone() for x in out]
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, out):
            assert torch.equal(x, y) and torch.isfinite(x).all() and x.abs().max() > 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", [(1, 8, 16), (150, 72, 40), (300, 520, 264), (2500, 64, 128)], ids=lambda s: "x".join(map(str, s)))
def test_the_workspace_is_as_large_as_its_query_says(shape, dtype):
    """Both directions with exactly the queried bytes, inside a larger buffer whose other bytes stay as they were."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    m, n, k = shape
    H.note(f"gated workspace {shape} {dtype}")
    a, wg, wu, dh = (x.cuda() for x in _data(m, n, k, dtype, 1))
    out = [torch.zeros(m, n, dtype=a.dtype, device="cuda") for _ in range(3)]
    grads = [torch.zeros_like(a)] + [torch.zeros(n, k, device="cuda") for _ in range(2)]
    pad = 1 << 16
    for backward in (False, True):
        need = (B.gated_backward_workspace if backward else B.gated_project_workspace)(a.dtype, m, n, k)
        buf = torch.full((pad + need + pad,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = buf[pad:pad + need] if need else None
        if backward:
            B.gated_backward(dh, out[1], out[2], a, wg, wu, *grads, workspace=ws)
        else:
            B.gated_project(a, wg, wu, out[0], gate=out[1], up=out[2], workspace=ws)
        assert (buf[:pad] == 0xA5).all() and (buf[pad + need:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", [(1, 64, 256), (3, 200, 72), (8, 72, 520)], ids=lambda s: "x".join(map(str, s)))
def test_weight_gradients_are_float32_results(shape, dtype):
    """With few rows the bound on a weight gradient is close enough to show a part of dG or dU that does not reach the products:
    16 u of |dH U| (1 + |G|) or |dH| (1 + |G|) as above, 2^-23 for float32's dropped part products, 2^-22 of a term or 2^-39 of its
    column's largest for f16's two scaled parts, and the sums' 2 (m + 8) u.  Two parts of bf16 break it."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    m, n, k = shape
    H.note(f"gated float32 weight gradients {shape} {dtype}")
    a, wg, wu, dh = _data(m, n, k, dtype, 21)
    rng = np.random.default_rng(22)
    gate, up = (torch.from_numpy((1 + np.abs(rng.standard_normal((m, n)))).astype(np.float32)).to(a.dtype) for _ in range(2))
    dw = [torch.full((n, k), float("nan"), device="cuda") for _ in range(2)]
    B.gated_backward(*(x.cuda() for x in (dh, gate, up, a, wg, wu)), None, *dw, act=2,
                     workspace=_space(B.gated_backward_workspace(a.dtype, m, n, k)))
    aa, fdh, fg, fu = (_np(x) for x in (a, dh, gate, up))
    for name, got, d, own in (("dwg", dw[0], fdh * fu * T.act_slope(fg, "silu"), fdh * fu * (1 + fg)),
                              ("dwu", dw[1], fdh * T.act(fg, "silu"), fdh * (1 + fg))):
        t = np.abs(d)
        e = 16 * U * np.abs(own) + (2 + 2 * (m + 8)) * U * t
        if dtype == "float16":
            e = e + 2.0 ** -22 * t + 2.0 ** -39 * t.max(0)
        bound = e.T @ np.abs(aa)
        err = np.abs(_np(got) - d.T @ aa)
        assert (err <= bound).all(), (name, float((err / bound).max()))
        if dtype == "bfloat16" and m == 1:
            first = torch.from_numpy(d).to(torch.bfloat16).double()
            two = (first + (torch.from_numpy(d) - first).to(torch.bfloat16).double()).numpy()
            assert (np.abs(two.T @ aa - d.T @ aa) > bound).any()


def test_bf16_gradients_at_the_end_of_the_range():
    """An infinite dH makes its column's weight gradients infinite with A's signs; a dgate between bf16's and float32's
    largest values stays finite."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    m, n, k = 5, 16, 8
    H.note("gated bf16 range")
    a, wg, wu, dh = _data(m, n, k, "bfloat16", 5)
    a[2] = torch.tensor([0.25, -0.5, 0.125, -0.0625, 0.25, -0.25, 0.5, -0.125])
    gate, up = torch.full((m, n), 2.0, dtype=torch.bfloat16), torch.full((m, n), 3.0, dtype=torch.bfloat16)
    dh[2, 11] = float("inf")
    dh[2, 9], up[2, 9], gate[2, 9] = 1.4140625 * 2.0 ** 64, 1.4140625 * 2.0 ** 63, 0.0    # dgate 1.99957 2^127, bf16 ends at 1.99219 2^127
    dw = [torch.zeros(n, k, device="cuda") for _ in range(2)]
    B.gated_backward(*(x.cuda() for x in (dh, gate, up, a, wg, wu)), None, *dw, act=0,
                     workspace=_space(B.gated_backward_workspace(torch.bfloat16, m, n, k)))
    got = _np(dw[0])
    assert (got[11] == np.inf * np.sign(_np(a)[2])).all() and (_np(dw[1])[11] == got[11]).all()
    with np.errstate(over="ignore", invalid="ignore"):
        d = _np(dh) * _np(up)
    rest = np.arange(n) != 11
    assert d[2, 9] > 3.3895313892515355e38
    ref = d[:, rest].T @ _np(a)
    bound = (2 + 2 * (m + 8)) * U * (np.abs(d[:, rest]).T @ np.abs(_np(a)))
    assert (np.abs(got[rest] - ref) <= bound).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_one_row_of_a_buffer_with_odd_rows(dtype):
    """A single row may lie anywhere that is aligned: the stride to a next one that is not there does not count."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.note(f"gated one row of odd rows {dtype}")
    a, wg, wu, _ = (x.cuda() for x in _data(1, 64, 72, dtype, 3))
    h, _, _ = _forward(a, wg, wu, "silu", kept=False)
    wide = torch.full((2, 79), 5.0, dtype=a.dtype, device="cuda")
    wide[:1, :72] = a
    out = torch.full((2, 67), 5.0, dtype=a.dtype, device="cuda")
    B.gated_project(wide[:1, :72], wg, wu, out[:1, :64])
    assert torch.equal(out[:1, :64], h) and (out[:, 64:] == 5).all() and (out[1] == 5).all()
    y = torch.empty_like(h)
    B.group_norm_fwd(h, y, 4)
    B.group_norm_fwd(out[:1, :64], out[:1, :64], 4)
    assert torch.equal(out[:1, :64], y)
