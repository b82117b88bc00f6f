"""qha_newton_schulz and qha_muon_step against the float64 oracle.

Tolerances, u = 2^-24.  A stored value (X, A or B) is within 4 u of itself, a term of a product within 12 u (two operands and
the dropped product of their second parts), and a sum of n terms passes at most 3 n + 16 float32 additions.  So one step
with one coefficient is checked value by value against the same products of magnitudes: A is off by (3 n + 28) u |X| |X|^T, and
so on (`_one_step`, which also counts the half step 2^-25 of second parts that are subnormal in half precision).  These bounds grow with n, rounding errors mostly cancel: over all values, the root mean square of error over
magnitude must stay below 16 u (12 u of the operands at worst, and 4).
Over several steps errors grow by at most L = 4.3 a step, the largest slope of s -> 3.4445 s - 4.775 s^3 + 2.0315 s^5 and of its
quotient by s on [0, 1.21].  A step's own error, on the root mean square, is at most 20 (the sum of the sizes of a X, b A X and c A A X,
each twice) times sqrt(3 n / 16 + 16) u of X's norm: matrix cores add 16 terms at a time.  So O is off by the sum over steps k of
L^(4 - k) 20 sqrt(3 n / 16 + 16) u |X_k| in norm (`_five_steps`).
"""
import numpy as np
import pytest

import gpu_helpers as H
from oracle import train as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 0.0, "bfloat16": 0.0, "float16": 2.0 ** -25}
FIVE = [(3.4445, -4.7750, 2.0315)] * 5
L = 4.3

# on chip: a value, a row, a column, odd sizes, whole blocks of 32, the longest; tiles: just over it, odd, whole, long, tall
SMALL = [(1, 1), (1, 7), (7, 1), (16, 16), (33, 20), (31, 128), (128, 100), (97, 97), (128, 128), (128, 1), (64, 127),
         (129, 1), (1, 129), (130, 64), (32, 896), (895, 3), (33, 384), (380, 64), (65, 65), (96, 192), (190, 70), (5, 65)]
LARGE = [(897, 1), (1, 900), (385, 64), (64, 200), (193, 193), (256, 256), (333, 777), (1000, 520), (5, 3001), (700, 12), (512, 512)]


def _draw(shape, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal(shape) * scale).astype(np.float32)


def _t(a, dtype="float32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, dtype)).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _run(xs, steps, out_dtype="float32", eps=1e-7, outs=None):
    """One call over the list of GPU matrices."""
    import torch
    from quantized_halo_aggregation_amd import binding as B
    if outs is None:
        outs = [torch.full_like(x, float("nan"), dtype=getattr(torch, out_dtype)) for x in xs]
    ws = torch.empty(max(B.newton_schulz_workspace([tuple(x.shape) for x in xs], len(steps)), 16), dtype=torch.uint8,
                     device="cuda")
    B.newton_schulz(xs, outs, steps=len(steps), coefficients=steps, eps=eps, workspace=ws)
    return outs


def _one_step(got, x, abc, eps):
    """Every value of one step's result `got` for x: float64 tensors on the GPU."""
    a, b, c = abc
    x = x / ((x * x).sum().sqrt() + eps)
    x = x if x.shape[0] <= x.shape[1] else x.T.contiguous()
    got = got if got.shape == x.shape else got.T
    m, n = x.shape
    g = lambda k: (3 * k + 20) * U          # the additions, and the dropped product of second parts
    tiny = 2.0 ** -37                       # half a step of subnormal second parts, after scaling by 4096
    ax = x.abs()
    # a stored value is off by 4 u of itself and by `tiny` where it is small: x enters a x, the gram product (twice)
    # and B x with that error
    dx = 4 * U * ax + tiny
    s, ms = x @ x.T, ax @ ax.T
    es = 2 * dx @ (ax + dx).T + g(n) * ms + 4 * U * s.abs() + tiny
    es = es.maximum(es.T)
    w, ma = b * s + c * s @ s, s.abs() + es
    mw = abs(b) * ma + abs(c) * ma @ ma
    ew = abs(b) * es + abs(c) * (2 * es @ ma + g(m) * ma @ ma) + 8 * U * mw + 4 * tiny
    ref = a * x + w @ x
    bound = abs(a) * dx + ew @ (ax + dx) + mw @ dx + g(m) * mw @ ax + 8 * U * (abs(a) * ax + ref.abs()) + tiny
    err = (got - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    # magnitudes of the whole step, with which errors that do not cancel would grow; x and the result are also off by up to
    # `tiny` each, whatever their size, which would be any share of a value near zero: that much is not counted
    size = abs(a) * ax + mw @ ax
    err = (err - (abs(a) + 1) * tiny).clamp(min=0)
    assert float(((err / size) ** 2).mean()) ** 0.5 <= 16 * U * (1 + (b != 0) + 3 * (c != 0))


def _five_steps(got, x, dtype, eps=1e-7, steps=FIVE):
    ref = T.newton_schulz(x, steps, eps)
    _, s, _ = np.linalg.svd(x / (np.sqrt((x * x).sum()) + eps), full_matrices=False)
    bound = 0.0
    for k, (a, b, c) in enumerate(steps):
        bound += L ** (len(steps) - 1 - k) * 20 * np.sqrt(3 * max(x.shape) / 16 + 16) * U * np.sqrt((s * s).sum())
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.isfinite(got).all()
    off = np.abs(got - ref)
    assert np.sqrt((np.maximum(off - HALF[dtype] * np.abs(got) * (1 + HALF[dtype]) - TINY[dtype], 0) ** 2).sum()) <= bound
    # the float32 result itself is far better than that in practice: a lost second part would leave 2^-12 of X
    if dtype == "float32":
        assert np.sqrt((off ** 2).sum()) <= 2.0 ** -12 * np.sqrt((ref ** 2).sum())


@pytest.mark.parametrize("abc", [(2.0, 0.0, 0.0), (0.0, 3.0, 0.0), (0.0, 0.0, -2.0), (3.4445, -4.7750, 2.0315)],
                         ids=["own", "cubic", "quintic", "all"])
@pytest.mark.parametrize("shape", SMALL + LARGE, ids=lambda s: "x".join(map(str, s)))
def test_one_step_value_by_value(shape, abc):
    H.require_gpu()
    H.note(f"newton-schulz one step {shape} {abc}")
    x = _draw(shape, 1, 1e-3)
    out, = _run([_t(x)], [abc])
    _one_step(out.double(), _t(x).double(), abc, 1e-7)


@pytest.mark.parametrize("types", [("float32", "float32"), ("bfloat16", "float32"), ("float16", "float16"),
                                   ("bfloat16", "bfloat16"), ("float32", "float16")], ids="-".join)
def test_five_steps_of_a_mixed_list(types):
    """Every size in one call: small and tiled ones, more than a batch's table holds."""
    H.require_gpu()
    H.note(f"newton-schulz five steps {types}")
    xs = [_t(_draw(s, 10 + i, 0.01), types[0]) for i, s in enumerate((SMALL + LARGE) * 3)]
    for x, o in zip(xs, _run(xs, FIVE, types[1])):
        _five_steps(_np(o), _np(x), types[1])


def test_many_tiles():
    """Enough tiles for the larger ones: eight of 1000 x 1100 and, apart, a wide and a tall one of 1500 x 2100."""
    H.require_gpu()
    H.note("newton-schulz many tiles")
    xs = [_t(_draw((1000, 1100), 30 + i)) for i in range(8)]
    outs = _run(xs, FIVE)
    for i in (0, 7):
        _five_steps(_np(outs[i]), _np(xs[i]), "float32")
    again = _run(xs[3:4], FIVE)[0]
    _five_steps(_np(again), _np(xs[3]), "float32")
    x = _draw((1500, 2100), 50)
    wide, tall = _run([_t(x)], FIVE)[0], _run([_t(x.T)], FIVE)[0]
    _five_steps(_np(wide), x.astype(np.float64), "float32")
    assert bool((wide == tall.T).all())


def _products(got, x, dtype="float32", eps=1e-7):
    """_five_steps for large matrices: the same bound, with the steps as products in float64 on the GPU in the
    place of singular values (their sum of squares is X's)."""
    x = x.double()
    got = got.double() if x.shape[0] <= x.shape[1] else got.double().T
    x = x if x.shape[0] <= x.shape[1] else x.T.contiguous()
    x = x / ((x * x).sum().sqrt() + eps)
    bound = 0.0
    for k, (a, b, c) in enumerate(FIVE):
        bound += L ** (4 - k) * 20 * np.sqrt(3 * x.shape[1] / 16 + 16) * U * float((x * x).sum()) ** 0.5
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    off = (got - x).abs()
    assert bool(got.isfinite().all())
    assert float(((off - HALF[dtype] * got.abs() * (1 + HALF[dtype]) - TINY[dtype]).clamp(min=0) ** 2).sum()) ** 0.5 <= bound
    if dtype == "float32":
        assert float((off * off).sum()) <= 2.0 ** -24 * float((x * x).sum())


# the rule on tiles takes sides of 64, of which each half of the reduction is a group's own (one of 1001 x 1300 in its A; 1000 x 900 with
# 29 steps, and 30 x 1000 with one beside it), of 128 (one of 2501 x 3001), 192 and 256 (one of 4001 x 4090) and 256 (24 of 1000 x 4070)
LARGER = [[(1001, 1300)], [(1000, 900), (30, 1000)], [(2501, 3001)], [(3001, 2501)], [(4001, 4090)], [(4090, 4001)], [(1000, 4070), (4070, 1000)] * 12,
          [(1024, 4096)] * 24]


def _on_gpu(shapes, seed, dtype="float32", scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=gen, device="cuda") * scale).to(getattr(torch, dtype)) for s in shapes]


@pytest.mark.parametrize("shapes", LARGER, ids=lambda s: f"{len(s)}of" + "x".join(map(str, s[0])))
def test_larger_tiles(shapes):
    """One step value by value, and five."""
    H.require_gpu()
    H.note(f"newton-schulz larger tiles {len(shapes)} of {shapes[0]}")
    xs = _on_gpu(shapes, 5)
    outs = _run(xs, FIVE[:1])
    for i in sorted({0, len(xs) // 2, len(xs) - 1}):
        _one_step(outs[i].double(), xs[i].double(), FIVE[0], 1e-7)
    outs = _run(xs, FIVE, "float16")
    for i in sorted({0, len(xs) - 1}):
        _products(outs[i], xs[i], "float16")


@pytest.mark.parametrize("shapes", [[(96, 2848)] * 12, [(100, 1000), (1000, 90)], [(130, 150), (40, 2000), (300, 20)],
                                    [(33 + i, 901 - i) for i in range(45)]],
                         ids=["many-96", "two-of-128-rows", "mixed", "more-than-a-batch"])
def test_blocks_straight_from_memory(shapes):
    """B's rows formed by the last product's blocks or by a launch of its own, and lists of more than one batch."""
    H.require_gpu()
    H.note(f"newton-schulz from memory {len(shapes)} of {shapes[0]}")
    xs = _on_gpu(shapes, 6)
    one, five = _run(xs, FIVE[:1]), _run(xs, FIVE)
    for x, o, f in zip(xs, one, five):
        _one_step(o.double(), x.double(), FIVE[0], 1e-7)
        _products(f, x)


def test_rows_far_apart():
    """Offsets past 2^31 elements, of the source and of the result: on chip (800 x 30) and tiled (1100 x 300)."""
    import torch
    H.require_gpu()
    H.note("newton-schulz rows far apart")
    for rows, cols in ((800, 30), (1100, 300)):
        ld = (2 ** 31 + 2 ** 28) // rows
        x, = _on_gpu([(rows, cols)], 8, "bfloat16")
        want, = _run([x], FIVE, "bfloat16")
        buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
        view = buf.view(rows, ld)[:, ld - cols:]
        view.copy_(x)
        _run([view], FIVE, outs=[view])
        assert torch.equal(view, want)
        del buf, view


def test_a_matrix_does_not_depend_on_its_neighbours():
    """Bit by bit on what the others hold; on their sizes only by how its sums are cut, and not at all on chip."""
    import torch
    H.require_gpu()
    H.note("newton-schulz alone and among others")
    shapes = [(100, 90), (200, 300), (300, 200), (64, 64), (400, 130)]
    xs = [_t(_draw(s, 60 + i)) for i, s in enumerate(shapes)]
    together = _run(xs, FIVE)
    for i, (x, o) in enumerate(zip(xs, together)):
        others = [x if k == i else _t(_draw(s, 160 + k)) for k, s in enumerate(shapes)]
        assert torch.equal(_run(others, FIVE)[i], o)
        alone, = _run([x], FIVE)
        _five_steps(_np(alone), _np(x), "float32")
        assert max(x.shape) > 128 or torch.equal(alone, o)
    assert all(torch.equal(a, b) for a, b in zip(_run(xs, FIVE), together))


@pytest.mark.parametrize("shape", [(60, 50), (200, 330)])
def test_strided_rows_odd_offsets_and_in_place(shape):
    import torch
    H.require_gpu()
    H.note(f"newton-schulz strided {shape}")
    x = _t(_draw(shape, 70))
    plain, = _run([x], FIVE)
    for extra, dtype in ((3, "float32"), (8, "float32"), (1, "bfloat16")):
        src = x.to(getattr(torch, dtype))
        want, = _run([src], FIVE)
        buf = torch.full((shape[0], shape[1] + 2 * extra), 9.0, dtype=src.dtype, device="cuda")
        view = buf[:, extra:-extra]
        view.copy_(src)
        res = torch.full((shape[0] + 2, shape[1] + extra), 9.0, device="cuda")
        out = res[1:-1, :shape[1]]
        _run([view], FIVE, outs=[out])
        assert torch.equal(out, want)
        assert bool((res[0] == 9).all()) and bool((res[-1] == 9).all()) and bool((res[:, shape[1]:] == 9).all())
        assert bool((buf[:, :extra] == 9).all()) and bool((buf[:, -extra:] == 9).all())
    own = x.clone()
    _run([own], FIVE, outs=[own])
    assert torch.equal(own, plain)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_any_size_of_gradient(scale):
    """The norm is summed in float64, so that squares neither overflow nor vanish."""
    H.require_gpu()
    H.note(f"newton-schulz scale {scale}")
    for shape in ((50, 60), (150, 180)):
        x = _draw(shape, 80) * np.float32(scale)
        out, = _run([_t(x)], FIVE, eps=0.0)
        _five_steps(_np(out), x.astype(np.float64), "float32", eps=0.0)


def test_zeros_and_values_that_are_not_finite():
    import torch
    H.require_gpu()
    H.note("newton-schulz special values")
    for shape in ((50, 60), (150, 180)):
        good = _t(_draw(shape, 90))
        want, = _run([good], FIVE)
        bad = []
        for value in (float("nan"), float("inf"), float("-inf")):
            bad.append(good.clone())
            bad[-1][7, 5] = value
        for eps in (0.0, 1e-7):
            outs = _run([bad[0], good, bad[1], torch.zeros(shape, device="cuda"), bad[2]], FIVE, eps=eps)
            assert all(bool(torch.isnan(outs[i]).all()) for i in (0, 2, 4))
            assert bool((outs[3] == 0).all())
            assert bool(torch.isfinite(outs[1]).all()) and (eps == 0.0 or torch.equal(outs[1], want))
    # one row that is not zero stays the only one
    x = torch.zeros(140, 150, device="cuda")
    x[17] = 1.0
    out, = _run([x], FIVE)
    assert bool((out[:17] == 0).all()) and bool((out[18:] == 0).all()) and bool((out[17] != 0).all())
    _five_steps(_np(out), _np(x), "float32")


def test_orthonormal_rows_come_out_of_cubic_steps():
    """Sixteen steps of 1.5 s - 0.5 s^3 from singular values in [0.05, 0.3]: X X^T is the unit matrix to 2e-5."""
    H.require_gpu()
    H.note("newton-schulz orthonormal rows")
    rng = np.random.default_rng(4)
    for m, n in ((40, 90), (160, 200)):
        q, _ = np.linalg.qr(rng.standard_normal((n, m)))
        r, _ = np.linalg.qr(rng.standard_normal((m, m)))
        x = (r * rng.uniform(0.5, 3, m)) @ q.T
        out, = _run([_t(x.astype(np.float32))], [(1.5, -0.5, 0.0)] * 16)
        # values from 0.5 / (3 sqrt(160)) = 0.013 grow 1.5 a step: 16 steps reach 1; the last steps lose their own rounding alone
        assert np.abs(_np(out) @ _np(out).T - np.eye(m)).max() < 2e-5


# ---------------------------------------------------------------------------------------------
# the optimiser
# ---------------------------------------------------------------------------------------------

def _muon_case(shapes, grad, copy, seed=3, **kw):
    import torch
    from quantized_halo_aggregation_amd import binding as B
    params = [_t(_draw(s, seed + i, 0.1)) for i, s in enumerate(shapes)]
    momenta = [_t(_draw(s, seed + 100 + i, 0.02)) for i, s in enumerate(shapes)]
    grads = [_t(_draw(s, seed + 200 + i, 0.01), grad) for i, s in enumerate(shapes)]
    copies = [torch.full_like(p, float("nan"), dtype=getattr(torch, copy)) for p in params] if copy else None
    return B.Muon(params, momenta=momenta, copies=copies, **kw), grads


SHAPES = [(40, 40), (128, 128), (1, 9), (100, 30), (200, 150), (130, 400), (333, 70), (256, 256)]


@pytest.mark.parametrize("grad,copy,nesterov,scale", [("float32", None, True, "spectral"), ("bfloat16", "bfloat16", True, "rms"),
                                                      ("float16", "float32", False, 0.7), ("float32", "float16", False, "rms")])
def test_muon_steps(grad, copy, nesterov, scale):
    """Three steps, each from the library's own state.  The momentum passes three roundings, the parameter three and
    lr scale times O's error, which is bounded as above."""
    H.require_gpu()
    H.note(f"muon {grad} {copy} nesterov {nesterov} {scale}")
    opt, grads = _muon_case(SHAPES, grad, copy, nesterov=nesterov, scale=scale, weight_decay=0.1, momentum=0.9)
    for turn in range(3):
        before = [(_np(p), _np(m)) for p, m in zip(opt.params, opt.m)]
        opt.step(grads, 0.05, grad_scale=0.5 + turn)
        for i, s in enumerate(SHAPES):
            p, m = before[i]
            size = {"spectral": max(1.0, s[0] / s[1]) ** 0.5, "rms": 0.2 * max(s) ** 0.5}.get(scale, scale)
            g = _np(grads[i])
            mu = np.float64(np.float32(0.9))
            want_p, want_m = T.muon(p, g, m, 0.05, mu, nesterov, 0.1, size, 0.5 + turn, FIVE, 1e-7)
            assert (np.abs(_np(opt.m[i]) - want_m) <= 3 * U * (np.abs(mu * m) + np.abs((0.5 + turn) * g))).all()
            u = (0.5 + turn) * g + mu * want_m if nesterov else want_m
            s_k = np.linalg.svd(u / (np.sqrt((u * u).sum()) + 1e-7), compute_uv=False)
            bound = L ** 5 * 6 * U * np.sqrt((s_k * s_k).sum())                       # u's own roundings
            for k, (a, b, c) in enumerate(FIVE):
                bound += L ** (4 - k) * 20 * np.sqrt(3 * max(s) / 16 + 16) * U * np.sqrt((s_k * s_k).sum())
                s_k = a * s_k + b * s_k ** 3 + c * s_k ** 5
            off = np.abs(_np(opt.params[i]) - want_p) - 3 * U * (np.abs(p) + np.abs(want_p))
            assert np.sqrt((np.maximum(off, 0) ** 2).sum()) <= 0.05 * size * bound
            if copy:
                assert bool((opt.copies[i] == opt.params[i].to(opt.copies[i].dtype)).all())


def test_muon_is_the_same_as_its_parts():
    """The step's O is that of newton_schulz for the momentum it leaves: p = decay p - step O."""
    import torch
    H.require_gpu()
    H.note("muon against newton-schulz")
    opt, grads = _muon_case(SHAPES, "float32", None, nesterov=False, scale=1.0, weight_decay=0.0)
    before = [p.clone() for p in opt.params]
    opt.step(grads, 1.0)
    for p, m, q, o in zip(before, opt.m, opt.params, _run(opt.m, FIVE)):
        assert bool(((p - o - q).abs() <= 2 * U * (p.abs() + o.abs())).all())
    opt, _ = _muon_case(SHAPES, "float32", None, nesterov=False, scale=1.0, weight_decay=0.5)
    before = [p.clone() for p in opt.params]
    opt.step([torch.zeros_like(p) for p in before], 0.0)
    assert all(torch.equal(p, q) for p, q in zip(before, opt.params))


@pytest.mark.parametrize("shapes,copy", [([(1024, 4096), (4096, 1024)] * 6, "bfloat16"), ([(1000, 4070)] * 3, "float16"),
                                         ([(2496, 3008)], None), ([(2501, 3004)], "float32")],
                         ids=["whole-blocks", "odd-rows", "one", "ragged"])
def test_muon_at_larger_tiles(shapes, copy):
    """As above, for the weights' and the copies' paths out of the tiled products."""
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.require_gpu()
    H.note(f"muon larger tiles {len(shapes)} of {shapes[0]} {copy}")
    params, grads = _on_gpu(shapes, 11, scale=0.1), _on_gpu(shapes, 12, "bfloat16", 0.01)
    copies = [torch.full_like(p, float("nan"), dtype=getattr(torch, copy)) for p in params] if copy else None
    opt = B.Muon(params, nesterov=False, scale=0.5, weight_decay=0.25, copies=copies)
    before = [p.clone() for p in params]
    opt.step(grads, 0.5)
    assert all(torch.equal(m, g.float()) for m, g in zip(opt.m, grads))
    for i, (p, q, o) in enumerate(zip(before, opt.params, _run(opt.m, FIVE))):
        want = p.double() * (1 - 0.125) - o.double() * 0.25
        assert bool(((want - q).abs() <= 3 * U * (p.abs() + o.abs())).all())
        assert copy is None or torch.equal(copies[i], q.to(copies[i].dtype))


def test_a_bad_gradient_spoils_its_own_matrix_alone():
    import torch
    H.require_gpu()
    H.note("muon bad gradient")
    good, grads = _muon_case(SHAPES, "float32", None)
    good.step(grads, 0.1)
    opt, grads = _muon_case(SHAPES, "float32", None)
    grads[1][3, 3] = float("nan")
    grads[5][100, 399] = float("inf")
    opt.step(grads, 0.1)
    for i in range(len(SHAPES)):
        if i in (1, 5):
            assert bool(torch.isnan(opt.params[i]).all())
        else:
            assert torch.equal(opt.params[i], good.params[i]) and torch.equal(opt.m[i], good.m[i])


def test_muon_on_another_stream_replayed_and_resumed():
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.require_gpu()
    H.note("muon streams, graphs, resume")
    eager, grads = _muon_case(SHAPES, "bfloat16", "bfloat16")
    opt, _ = _muon_case(SHAPES, "bfloat16", "bfloat16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step(grads, 0.1)
    torch.cuda.current_stream().wait_stream(side)
    eager.step(grads, 0.1)
    same = lambda: all(torch.equal(a, b) for a, b in zip(opt.params + opt.m + opt.copies, eager.params + eager.m + eager.copies))
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grads, 0.1)
    for turn in range(4):
        for i, g in enumerate(grads):
            g.copy_(torch.randn(g.shape, device="cuda") * 0.01 * (turn + 1))
        graph.replay()
        torch.cuda.synchronize()
        eager.step(grads, 0.1)
        assert same(), turn
    # a resume: new parameters and momenta with the saved values
    again = B.Muon([p.clone() for p in eager.params], momenta=[m.clone() for m in eager.m])
    again.step(grads, 0.1)
    eager.step(grads, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(again.params + again.m, eager.params + eager.m))
