"""qha_newton_schulz where values are of very different sizes: rows and columns that fade by 1e-6, singular values that
fall by 1e-4 and more, and steps that shrink X.

Tolerances, u = 2^-24.  X, A and B are held as two half-precision parts under a power of two that takes their bound (1 for the
first X, the largest value of the polynomials behind it; for A its square; for B the largest a + b s^2 + c s^4) to between 30000
and 60000: a value is within 4 u of itself or, where its second part is subnormal, 2^-25 / 30000 < 2^-39.8 (FLOOR) of the
bound.  A term of a product is off by 12 u (two operands and the dropped product of their second parts) and passes
at most 3 n + 16 float32 additions in a sum of n terms.
"""
import numpy as np
import pytest

import gpu_helpers as H
from test_gpu_newton_schulz import FIVE, U, _on_gpu, _products, _run

pytestmark = pytest.mark.gpu
FLOOR = 2.0 ** -39.8
# on chip (32, 64, 96 and 128 rows), blocks straight from memory with B's rows formed there and before, tiles of 64 (halves of the
# reduction and whole), 128 and 256
SHAPES = [(30, 800), (64, 380), (190, 96), (128, 128), (100, 700), (300, 200), (1000, 1000), (1300, 1700), (2400, 2600), (4001, 4090)]


def _graded(shape, how, seed=3):
    """Noise whose rows, columns or both fade to 1e-6, on the GPU."""
    import torch
    x, = _on_gpu([shape], seed)
    fade = lambda n: torch.logspace(0, -6, n, device="cuda")
    if how in ("rows", "both"):
        x = x * fade(shape[0])[:, None]
    if how in ("columns", "both"):
        x = x * fade(shape[1])
    return x


def _bounds(steps):
    """The largest singular value before each step and behind the last, and the largest of each a + b s^2 + c s^4."""
    r = np.linspace(0, 1, 100001)
    tops, inners = [1.0], []
    for a, b, c in steps:
        s = tops[-1] * r
        inners.append(np.abs(a + b * s ** 2 + c * s ** 4).max())
        tops.append(np.abs(s * (a + b * s ** 2 + c * s ** 4)).max())
    return tops, inners


@pytest.mark.parametrize("how", ["rows", "columns", "both"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_one_step_of_faded_values(shape, how):
    """Value by value.  a X goes through the last product, whose additions it passes."""
    H.require_gpu()
    H.note(f"newton-schulz faded {how} {shape}")
    given = _graded(shape, how)
    got, = _run([given], FIVE[:1])
    a, b, c = FIVE[0]
    x, got = given.double(), got.double()
    if x.shape[0] > x.shape[1]:
        x, got = x.T.contiguous(), got.T.contiguous()
    x = x / ((x * x).sum().sqrt() + 1e-7)
    m, n = x.shape
    (_, top), (inner,) = _bounds(FIVE[:1])
    g = lambda k: (3 * k + 28) * U
    ax = x.abs()
    dx = 4 * U * ax + FLOOR
    s, ms = x @ x.T.contiguous(), ax @ ax.T.contiguous()
    es = 2 * dx @ (ax + dx).T.contiguous() + g(n) * ms + 4 * U * s.abs() + FLOOR
    es = es.maximum(es.T)
    w, ma = b * s + c * s @ s, s.abs() + es
    mw = abs(b) * ma + abs(c) * ma @ ma
    ew = abs(b) * es + abs(c) * (2 * es @ ma + g(m) * ma @ ma) + 8 * U * mw + inner * FLOOR
    ref = a * x + w @ x
    size = abs(a) * ax + mw @ ax
    bound = abs(a) * dx + ew @ (ax + dx) + mw @ dx + g(m) * size + 4 * U * ref.abs() + top * FLOOR
    err = (got - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("how", ["rows", "columns", "both"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_five_steps_of_faded_values(shape, how):
    """In norm, with the bound of equally sized noise."""
    H.require_gpu()
    H.note(f"newton-schulz five steps faded {how} {shape}")
    x = _graded(shape, how)
    _products(_run([x], FIVE)[0], x)


@pytest.mark.parametrize("fall", [4, 6])
@pytest.mark.parametrize("shape", SHAPES[:8], ids=lambda s: "x".join(map(str, s)))
def test_five_steps_of_a_steep_spectrum(shape, fall):
    """Singular values from 1 to 10^-fall, in norm."""
    import torch
    H.require_gpu()
    H.note(f"newton-schulz steep {fall} {shape}")
    k = min(shape)
    u, v = (torch.linalg.qr(t.double())[0] for t in _on_gpu([(shape[0], k), (shape[1], k)], 7))
    x = ((u * torch.logspace(0, -fall, k, dtype=torch.float64, device="cuda")) @ v.T.contiguous()).float()
    _products(_run([x], FIVE)[0], x)


def _term_by_term(x, steps):
    """The steps in float32, sums of products that are exact added one term after another."""
    import torch
    x = x if x.shape[0] <= x.shape[1] else x.T.contiguous()
    x = (x.double() / ((x.double() ** 2).sum().sqrt() + 1e-7)).float()

    def product(p, q):
        total = torch.zeros(p.shape[0], q.shape[1], device="cuda")
        for k in range(p.shape[1]):
            total = torch.addr(total.double(), p[:, k].double(), q[k].double()).float()
        return total
    for a, b, c in steps:
        s = product(x, x.T.contiguous())
        x = a * x + product(b * s + c * product(s, s), x)
    return x


@pytest.mark.parametrize("shape", SHAPES[:7], ids=lambda s: "x".join(map(str, s)))
def test_a_steep_spectrum_is_as_precise_as_float32(shape):
    """Singular values from 1 to 1e-4, where a X is most of most values: in norm no further off than float32 products
    that add one term after another, and a quarter of that for what two parts drop of each product."""
    import torch
    H.require_gpu()
    H.note(f"newton-schulz against float32 {shape}")
    k = min(shape)
    u, v = (torch.linalg.qr(t.double())[0] for t in _on_gpu([(shape[0], k), (shape[1], k)], 8))
    x = ((u * torch.logspace(0, -4, k, dtype=torch.float64, device="cuda")) @ v.T.contiguous()).float()
    got = _run([x], FIVE)[0]
    plain = _term_by_term(x, FIVE)
    y, got = (x, got) if shape[0] <= shape[1] else (x.T.contiguous(), got.T)
    y = y.double() / ((y.double() ** 2).sum().sqrt() + 1e-7)
    for a, b, c in FIVE:
        s = y @ y.T.contiguous()
        y = a * y + (b * s + c * s @ s) @ y
    off = lambda z: float((z.double() - y).norm() / y.norm())
    assert off(got) <= 1.25 * off(plain), (off(got), off(plain))


@pytest.mark.parametrize("shape", [(20, 50), (128, 100), (200, 300), (1000, 1100)], ids=lambda s: "x".join(map(str, s)))
def test_steps_that_shrink_x_keep_its_bits(shape):
    """X a_1 a_2 ..: every step has a bound of its own.  A step rounds twice, within 4 u, and drops as much; values are off by FLOOR of the
    step's bound, which the steps behind it scale as they do the bound: at most 7 times FLOOR of the last bound in all."""
    H.require_gpu()
    H.note(f"newton-schulz shrinking steps {shape}")
    x, = _on_gpu([shape], 9)
    y = x.double()
    y = y / ((y * y).sum().sqrt() + 1e-7)
    for own in ([1e-3] * 3, [0.02, 1e-4, 3.0], [1e-6, 50.0, 50.0], [1e-5] * 4):
        out, = _run([x], [(a, 0.0, 0.0) for a in own])
        want = y * float(np.prod(own))
        bound = 8 * U * (len(own) + 1) * want.abs() + 7 * FLOOR * float(np.prod(own))
        assert bool(((out.double() - want).abs() <= bound).all()), own


@pytest.mark.parametrize("shape", [(20, 50), (128, 100), (200, 300), (1000, 1100)], ids=lambda s: "x".join(map(str, s)))
def test_a_steep_fixed_point_stays_in_range(shape):
    """One value is its matrix's only singular value, 1, where 5 s - 20 s^3 + 16 s^5 has the slope 25: what rounding adds to it in a
    step, 2e-6 of its terms' 41, grows 25-fold in the next, and half precision's range must hold it."""
    import torch
    H.require_gpu()
    H.note(f"newton-schulz steep fixed point {shape}")
    xs = []
    for row, col in ((0, 0), (shape[0] - 1, 3), (7, shape[1] - 1)):
        xs.append(torch.zeros(shape, device="cuda"))
        xs[-1][row, col] = -3.7
    for x, out in zip(xs, _run(xs, [(5, -20, 16)] * 2, eps=0.0)):
        assert float((out - x.sign()).abs().max()) <= 2e-6 * 41 * 26


def test_steps_that_leave_nothing():
    """A step of zeros, and steps behind it, whatever they are."""
    import torch
    H.require_gpu()
    H.note("newton-schulz steps of zeros")
    for shape in ((30, 40), (200, 300), (1000, 1100)):
        x, = _on_gpu([shape], 10)
        for steps in ([(0, 0, 0)], [(0, 0, 0), FIVE[0], (1e-3, 1e30, -1e30)], [(1e-30, 0, 0), (1e-30, 0, 0), (0, 1e30, 0)]):
            out, = _run([x], steps)
            assert bool((out.abs() <= 1e-28).all()), steps


def test_muon_of_a_gradient_with_faded_rows():
    """The step's O is that of newton_schulz for the momentum it leaves, which the tests above check."""
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.require_gpu()
    H.note("muon faded rows")
    shapes = [(128, 128), (300, 200), (1000, 1100)]
    grads = [_graded(s, "rows") for s in shapes]
    params = [torch.zeros(s, device="cuda") for s in shapes]
    B.Muon(params, nesterov=False, scale=1.0).step(grads, 1.0)
    for p, o in zip(params, _run(grads, FIVE)):
        assert torch.equal(-p, o)
