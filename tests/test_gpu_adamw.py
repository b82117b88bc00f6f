"""qha_adamw_step and qha_adamw_values against the float64 oracle.

Tolerances count roundings, u = 2^-24 the unit roundoff of float32.  32-bit moments: the gradient
carries 2 (scale constant, product), each moment's products 2 (constant, product; one more for g^2,
which doubles the gradient's) and the sum 1, so m is off by at most 8 u (|b1 m| + |o1 g|) and v by
10 u v.  The parameter's update adds the root, two constants, three products, a sum and a quotient to
those: at most 24 u of step (|b1 m| + |o1 g|) / (c1 denominator); the decayed parameter is off by
4 u |p|.  8-bit moments are formed in float64 from g: codes are equal, and a scale is the float32
nearest to a float64 that may differ in its last bits (one float32 step).
"""
import numpy as np
import pytest

import gpu_helpers as H
from oracle import train as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = {"one": [1], "vectors": [1, 3, 0, 4, 255, 256, 257, 1023, 1024, 1025], "many": [5 + 7 * i for i in range(131)],
         "long": [70001, 3, 4096 * 5 + 2], "large": [(8 << 20) + 77]}


def _inputs(sizes, seed):
    rng = np.random.default_rng(seed)
    p = [rng.standard_normal(n).astype(np.float32) for n in sizes]
    g = [(rng.standard_normal(n) * 10.0 ** rng.uniform(-4, 0)).astype(np.float32) for n in sizes]
    m = [(rng.standard_normal(n) * 0.1).astype(np.float32) for n in sizes]
    v = [(rng.standard_normal(n) ** 2 * 0.01).astype(np.float32) for n in sizes]
    return p, g, m, v


def _cat(parts, starts, total):
    out = np.zeros(total, np.asarray(parts[0]).dtype if parts else np.float32)
    for x, s in zip(parts, starts):
        out[s:s + x.size] = x
    return out


def _check_param(got, p, m, v, mag, hyper, lr, step, extra=0.0):
    b1, b2, eps, wd = hyper
    ref = T.adam_param(p, m, v, lr, b1, b2, eps, wd, step)
    denom = np.sqrt(v / (1 - b2 ** step)) + eps
    bound = 4 * U * np.abs(p) + 24 * U * lr * mag / ((1 - b1 ** step) * denom) + extra
    assert (np.abs(got - ref) <= bound).all(), float((np.abs(got - ref) / bound).max())


@pytest.mark.parametrize("case", sorted(SIZES))
@pytest.mark.parametrize("gtype", ["float32", "bfloat16", "float16"])
def test_step_with_float32_moments(case, gtype):
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    sizes = SIZES[case]
    if case == "large" and gtype != "float32":
        pytest.skip("one large case is enough")
    p, g, m, v = _inputs(sizes, 1)
    b1, b2, eps, wd, lr, scale, t0 = 0.8, 0.98, 1e-6, 0.05, 3e-2, 0.7, 4
    dt = getattr(torch, gtype)
    H.note(f"adamw 32 {case} {gtype}")
    params = [H.dev(x) for x in p]
    copies = [torch.zeros(x.shape, dtype=dt, device="cuda") for x in params]
    opt = B.AdamW(params, bits=32, betas=(b1, b2), eps=eps, weight_decay=wd, copies=copies)
    opt.m.copy_(H.dev(_cat(m, opt.starts, opt.m.numel())))
    opt.v.copy_(H.dev(_cat(v, opt.starts, opt.v.numel())))
    opt.t = t0
    grads = [H.dev(x).to(dt) for x in g]
    opt.step(grads, lr, grad_scale=scale)
    assert opt.t == t0 + 1
    gm, gv = H.host(opt.m), H.host(opt.v)
    for i, s in enumerate(opt.starts):
        gi = grads[i].float().cpu().numpy().astype(np.float64) * scale
        rm, rv = T.adam_moments(m[i], v[i], gi, b1, b2)
        mag = b1 * np.abs(m[i]) + (1 - b1) * np.abs(gi)
        n = sizes[i]
        assert (np.abs(gm[s:s + n] - rm) <= 8 * U * mag).all()
        assert (np.abs(gv[s:s + n] - rv) <= 10 * U * rv + 1e-45).all()
        _check_param(H.host(params[i]), p[i], rm, rv, mag, (b1, b2, eps, wd), lr, t0 + 1)
        assert torch.equal(copies[i], params[i].to(dt))
    # nothing is written between the tensors
    inside = np.zeros(gm.size, bool)
    for s, n in zip(opt.starts, sizes):
        inside[s:s + n] = True
    assert (gm[~inside] == 0).all() and (gv[~inside] == 0).all()


@pytest.mark.parametrize("case", ["one", "vectors", "many", "long"])
@pytest.mark.parametrize("gtype", ["float32", "bfloat16"])
def test_steps_with_8_bit_moments(case, gtype):
    """Three steps from zero moments: every code equals the oracle's, which carries the GPU's scales
    into the next step."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    sizes = SIZES[case]
    p, _, _, _ = _inputs(sizes, 2)
    b1, b2, eps, wd, lr = 0.9, 0.999, 1e-8, 0.01, 1e-2
    H.note(f"adamw 8 {case} {gtype}")
    params = [H.dev(x) for x in p]
    opt = B.AdamW(params, bits=8, betas=(b1, b2), eps=eps, weight_decay=wd)
    for step in (1, 2, 3):
        _, g, _, _ = _inputs(sizes, 10 + step)
        grads = [H.dev(x).to(getattr(torch, gtype)) for x in g]
        before = [H.host(t).copy() for t in (opt.m, opt.v, opt.m_scale, opt.v_scale)]
        old = [H.host(t).copy() for t in params]
        opt.step(grads, lr)
        cm, cv, sm, sv = (H.host(t) for t in (opt.m, opt.v, opt.m_scale, opt.v_scale))
        vm, vv = (H.host(t) for t in opt.values())
        for i, s in enumerate(opt.starts):
            n = sizes[i]
            if n == 0:
                continue
            blk = slice(s // T.BLOCK, s // T.BLOCK + -(-n // T.BLOCK))
            gi = grads[i].float().cpu().numpy().astype(np.float64)
            om = T.decode(before[0][s:s + n], before[2][blk], 127, 2)
            ov = T.decode(before[1][s:s + n], before[3][blk], 255, 4)
            rm, rv = T.adam_moments(om, ov, gi, b1, b2)
            for got, scale, ref, top, power, values in ((cm, sm, rm, 127, 2, vm), (cv, sv, rv, 255, 4, vv)):
                codes, want = T.encode(ref, top, power)
                assert np.array_equal(got[s:s + n].astype(np.int64), codes)
                assert (np.abs(scale[blk].astype(np.float64) - want) <= 2 * U * want).all()
                back = T.decode(got[s:s + n], scale[blk], top, power)
                assert (np.abs(values[s:s + n] - back) <= 2 * U * np.abs(back)).all()
            mag = b1 * np.abs(om) + (1 - b1) * np.abs(gi)
            _check_param(H.host(params[i]), old[i], rm, rv, mag, (b1, b2, eps, wd), lr, step)


def test_codes_at_half_way_points_and_wide_ranges():
    """Moments that sit on, just under and just over the half-way points between codes, and a block
    that spans the whole float32 range: codes are those of the float64 decision."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    k = np.arange(127)
    half = ((k + 0.5) / 127) ** 2
    g = np.concatenate([[1.0], half, half * (1 + 1e-7), half * (1 - 1e-7), [0.0] * 130,
                        [3e19, 1e-30, -1e-38, 1e-45, 0.0, 5e18]]).astype(np.float32)
    H.note("adamw 8 half-way points")
    p = torch.zeros(g.size, device="cuda")
    opt = B.AdamW([p], bits=8, betas=(0.0, 0.5), weight_decay=0.0)
    opt.step([H.dev(g)], 1e-3)
    m, v = T.adam_moments(np.zeros(g.size), np.zeros(g.size), g, 0.0, 0.5)
    cm, sm = T.encode(m, 127, 2)
    cv, sv = T.encode(v, 255, 4)
    assert np.array_equal(H.host(opt.m).astype(np.int64)[:g.size], cm)
    assert np.array_equal(H.host(opt.v).astype(np.int64)[:g.size], cv)
    H.assert_bits_equal(H.host(opt.m_scale), sm)
    # 3e19 squared overflows float32: its block reads as NaN, the others do not
    assert np.isnan(sv).any() and np.array_equal(np.isnan(H.host(opt.v_scale)), np.isnan(sv))
    assert np.array_equal(np.isnan(H.host(opt.values()[1]))[:g.size], np.isnan(T.decode(cv, sv, 255, 4)))


def test_scales_and_codes_are_those_of_the_formula_as_written():
    """float64 moments from 16-bit gradients land half-way between two float32 scales in about one block of a hundred;
    the formula's products and sums, each rounded, decide there too: three steps stay bit for bit equal."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    n, rng = 400_000, np.random.default_rng(12)
    H.note("adamw 8 scales")
    opt = B.AdamW([torch.zeros(n, device="cuda")], bits=8)
    m, v, ms, vs = (np.zeros(n), np.zeros(n), np.zeros(-(-n // 256), np.float32), np.zeros(-(-n // 256), np.float32))
    wide = lambda s: np.repeat(s.astype(np.float64), 256)[:n]
    for _ in range(3):
        g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(torch.bfloat16)
        opt.step([g.cuda()], 1e-3)
        gd = g.float().numpy().astype(np.float64)
        x = 0.9 * ((wide(ms) * (m * np.abs(m))) * (1.0 / (127.0 * 127.0))) + (1.0 - 0.9) * gd
        y = 0.999 * ((wide(vs) * ((v * v) * (v * v))) * (1.0 / 255.0 ** 4)) + (1.0 - 0.999) * (gd * gd)
        (m, ms), (v, vs) = T.encode(x, 127, 2), T.encode(y, 255, 4)
        m, v = m.astype(np.float64), v.astype(np.float64)
        H.assert_bits_equal(H.host(opt.m_scale), ms, "m_scale")
        H.assert_bits_equal(H.host(opt.v_scale), vs, "v_scale")
        assert np.array_equal(H.host(opt.m)[:n], m) and np.array_equal(H.host(opt.v)[:n], v)


def test_codes_of_equal_and_zero_gradients():
    """Blocks whose largest magnitude is shared by many lanes, or is zero."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    g = np.zeros(1100, np.float32)
    g[256:512] = -0.3
    g[512:768:2] = 1e-3
    g[768:] = np.repeat(np.float32([1.0, -1.0, 0.25, 1e-30]), 83)
    H.note("adamw 8 equal gradients")
    opt = B.AdamW([torch.ones(1100, device="cuda")], bits=8)
    opt.step([H.dev(g)], 1e-3)
    m, v = T.adam_moments(np.zeros(1100), np.zeros(1100), g, 0.9, 0.999)
    for got, ref, top, power in ((opt.m, m, 127, 2), (opt.v, v, 255, 4)):
        assert np.array_equal(H.host(got).astype(np.int64)[:1100], T.encode(ref, top, power)[0])


@pytest.mark.parametrize("bits", [8, 32])
def test_a_gradient_that_is_not_finite(bits):
    """Only its own parameter is touched in that step; with 8-bit moments its block reads as NaN after."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    for bad in (np.inf, -np.inf, np.nan):
        H.note(f"adamw {bits} gradient {bad}")
        g = np.linspace(-1, 1, 700).astype(np.float32)
        g[300] = bad
        p = torch.ones(700, device="cuda")
        opt = B.AdamW([p], bits=bits)
        opt.step([H.dev(g)], 1e-3)
        got = H.host(p)
        assert np.isfinite(np.delete(got, 300)).all() and not np.isfinite(got[300])
        m, v = (H.host(t)[:700] for t in opt.values())
        hit = np.zeros(700, bool)
        hit[256:512] = True
        for x in (m, v):
            assert np.array_equal(np.isfinite(x), ~hit if bits == 8 else np.arange(700) != 300)


def test_unaligned_tensors_match_aligned_ones():
    """Views that start one element into a buffer take the element-wise accesses: same bits."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    n = 5003
    p, g, _, _ = _inputs([n], 5)
    for bits in (8, 32):
        H.note(f"adamw {bits} unaligned")
        out = []
        for off in (0, 1):
            buf = torch.zeros(n + off, device="cuda")
            cbuf = torch.zeros(n + off, dtype=torch.bfloat16, device="cuda")
            gbuf = torch.zeros(n + off, dtype=torch.bfloat16, device="cuda")
            buf[off:].copy_(H.dev(p[0]))
            gbuf[off:].copy_(H.dev(g[0]))
            opt = B.AdamW([buf[off:]], bits=bits, copies=[cbuf[off:]])
            for _ in range(2):
                opt.step([gbuf[off:]], 1e-2)
            out.append([H.host(t) for t in (buf[off:], cbuf[off:].float(), opt.m, opt.v)])
        for a, b in zip(*out):
            assert np.array_equal(a, b)


def test_step_on_another_stream_and_in_a_graph():
    """A captured step replays the launches: each replay equals an eager step at the same step number
    (the step number is a host value)."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    p, g, _, _ = _inputs([1000, 33], 7)
    H.note("adamw graph")
    side = torch.cuda.Stream()
    grads = [H.dev(x) for x in g]
    mk = lambda: B.AdamW([H.dev(x) for x in p], bits=8)
    eager, graphed = mk(), mk()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(grads, 1e-2)                     # eager, on the other stream
        graphed.t = 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            graphed.step(grads, 1e-2)
    torch.cuda.current_stream().wait_stream(side)
    eager.step(grads, 1e-2)
    for k in range(3):
        eager.t = 0
        eager.step(grads, 1e-2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.params + [eager.m, eager.v], graphed.params + [graphed.m, graphed.v]):
            assert torch.equal(a, b), k


def test_binding_refuses_gradients_that_do_not_fit():
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    p = torch.zeros(8, device="cuda")
    opt = B.AdamW([p])
    for bad, err in (([], ValueError), ([torch.zeros(7, device="cuda")], ValueError), ([torch.zeros(8)], ValueError),
                     ([torch.zeros(16, device="cuda")[::2]], ValueError),
                     ([torch.zeros(8, dtype=torch.float64, device="cuda")], TypeError)):
        with pytest.raises(err):
            opt.step(bad, 1e-3)
    with pytest.raises(ValueError, match="lr"):
        opt.step([p.clone()], -1.0)
    assert opt.t == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_replaced_tensors_are_the_ones_updated(bits):
    """A resume that assigns moments and replaces a parameter's .data goes on exactly as the run it came from, and
    leaves the tensors that were replaced alone."""
    H.require_gpu()
    import torch
    from quantized_halo_aggregation_amd import binding as B
    H.note(f"adamw {bits} resume")
    p, g, _, _ = _inputs([1000, 33], 9)
    grads = [H.dev(x) for x in g]
    names = ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ())
    run, resumed = (B.AdamW([H.dev(x) for x in p], bits=bits) for _ in range(2))
    run.step(grads, 1e-2)
    resumed.step(grads, 0.5)             # somewhere else: everything is replaced below
    old = [resumed.params[0].detach()] + [getattr(resumed, k) for k in names]
    kept = [t.clone() for t in old]
    for a, b in zip(resumed.params, run.params):
        a.data = b.clone()
    for k in names:
        setattr(resumed, k, getattr(run, k).clone())
    for _ in range(2):
        run.step(grads, 1e-2)
        resumed.step(grads, 1e-2)
    for a, b in zip(run.params + [getattr(run, k) for k in names], resumed.params + [getattr(resumed, k) for k in names]):
        assert torch.equal(a, b)
    for a, b in zip(old, kept):
        assert torch.equal(a, b)
