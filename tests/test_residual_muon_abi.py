"""Refusals of the entry points of the residual norm, Newton-Schulz and Muon, and of their binding, without a GPU.

Argument-error cases pass fake (never dereferenced) device addresses: the checks must fire first.
"""
import pytest
import torch

from quantized_halo_aggregation_amd import binding as B

FAKE = 0x10000
NAN = float("nan")


def _fwd(n=12, p=3, c=64, s=B.F32, t=B.F32, post=B.ROW_RMS, pre=B.ROW_LAYER, x=FAKE, ldx=64, h=FAKE, ldh=64, g=FAKE,
         ldg=64, pw=FAKE, pb=FAKE, qw=FAKE, qb=FAKE, skip=1.0, branch=1.0, eps=1e-6, y=FAKE, ldy=64, u=FAKE, ldu=64, ps=FAKE,
         qs=FAKE):
    return B._residual_norm_fwd(n, p, c, s, t, post, pre, x, ldx, h, ldh, g, ldg, pw, pb, qw, qb, skip, branch, eps, y, ldy,
                                u, ldu, ps, qs, None)


def _bwd(n=12, p=3, c=64, s=B.F32, t=B.F32, post=B.ROW_RMS, pre=B.ROW_LAYER, dy=FAKE, lddy=64, du=FAKE, lddu=64, y=FAKE,
         ldy=64, h=FAKE, ldh=64, g=FAKE, ldg=64, pw=FAKE, pb=FAKE, qw=FAKE, skip=1.0, branch=1.0, ps=FAKE, qs=FAKE, dx=FAKE,
         lddx=64, dh=FAKE, lddh=64, dg=FAKE, lddg=64, dpw=FAKE, dpb=FAKE, dqw=FAKE, dqb=FAKE, ws=FAKE, wsb=1 << 30):
    return B._residual_norm_bwd(n, p, c, s, t, post, pre, dy, lddy, du, lddu, y, ldy, h, ldh, g, ldg, pw, pb, qw, skip,
                                branch, ps, qs, dx, lddx, dh, lddh, dg, lddg, dpw, dpb, dqw, dqb, ws, wsb, None)


NO_BLOCK = dict(h=None, y=None, g=None, pw=None, pb=None, ps=None, post=B.ROW_NONE)
SHARED = [dict(n=-3), dict(n=1 << 31, p=1), dict(p=0), dict(n=10), dict(c=0), dict(c=66), dict(c=68, t=B.BF16), dict(s=3), dict(t=3),
          dict(s=B.BF16), dict(s=B.BF16, t=B.F16), dict(post=3), dict(pre=-1), dict(skip=NAN), dict(branch=float("inf")),
          dict(skip=1e300), dict(pw=FAKE + 4), dict(pb=FAKE + 8), dict(qw=FAKE + 4), dict(h=FAKE + 4), dict(ldh=60),
          dict(ldh=66), dict(g=FAKE + 8), dict(ldg=32), dict(post=B.ROW_NONE), dict(pre=B.ROW_NONE), dict(h=None),
          dict(ps=FAKE + 4), dict(qs=FAKE + 4)]


@pytest.mark.parametrize("bad", SHARED + [
    dict(x=None), dict(ldx=60), dict(x=FAKE + 4), dict(y=None), dict(y=FAKE + 8), dict(ldy=66), dict(u=None), dict(ldu=4),
    dict(qb=FAKE + 4), dict(eps=-1.0), dict(eps=NAN), dict(eps=1e300), dict(NO_BLOCK, y=FAKE), dict(NO_BLOCK, g=FAKE),
    dict(NO_BLOCK, pw=FAKE), dict(NO_BLOCK, post=B.ROW_RMS),
    dict(NO_BLOCK, pre=B.ROW_NONE, u=None, qs=None, qw=None, qb=None),
    dict(pre=B.ROW_NONE, qs=None, qw=None, qb=None), dict(pre=B.ROW_NONE, u=None, qs=None, qb=None),
    dict(s=B.F32, t=B.BF16, ldh=68)])
def test_residual_norm_fwd_refuses(bad):
    assert _fwd(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


@pytest.mark.parametrize("bad", SHARED + [
    dict(dy=FAKE + 4), dict(lddy=60), dict(du=None), dict(lddu=66), dict(y=None), dict(dx=None), dict(lddx=60),
    dict(dh=None), dict(dh=FAKE + 2), dict(dg=FAKE + 4), dict(g=None), dict(ps=None), dict(qs=None), dict(dpw=FAKE + 2),
    dict(dqb=FAKE + 1), dict(ws=FAKE + 8),
    dict(pre=B.ROW_NONE, dy=None, du=None, qs=None, qw=None, dqw=None, dqb=None),
    dict(NO_BLOCK, dh=None, dg=None, dpw=FAKE, dpb=None, y=FAKE), dict(NO_BLOCK, dg=None, dpw=None, dpb=None, y=FAKE)])
def test_residual_norm_bwd_refuses(bad):
    assert _bwd(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


def test_residual_norm_limits_and_workspace():
    wide = dict(c=8448, ldh=8448, ldg=8448, ldy=8448)
    assert _fwd(ldx=8448, ldu=8448, **wide) == B.QHA_ERR_UNSUPPORTED
    assert _bwd(lddx=8448, **wide) == B.QHA_ERR_UNSUPPORTED
    for sizes in ((0, 64), (-1, 64), (10, 8448), (10, 0), (10, 6)):
        assert B.residual_norm_workspace(*sizes) == 0
    assert B.residual_norm_workspace(10, 64, positions=3) == 0
    assert B.residual_norm_workspace(1, 4) >= 4 * 4 * 4          # one block's four vectors
    # a shared gate's partials come on top
    assert B.residual_norm_workspace(4096, 64, positions=4096) > B.residual_norm_workspace(4096, 64)
    assert _bwd(ws=None) == B.QHA_ERR_WORKSPACE
    assert _bwd(wsb=15) == B.QHA_ERR_WORKSPACE
    assert _fwd(n=0, x=None, y=None, h=None, u=None) == B.QHA_OK
    assert _bwd(n=0, dpw=None, dpb=None, dqw=None, dqb=None, dx=None) == B.QHA_OK


class Gpu(torch.Tensor):
    """A host tensor that says it lives on a GPU, so that what comes after that check is reached."""
    is_cuda = True
    index = 0

    def get_device(self):
        return type(self).index


class Other(Gpu):
    index = 1


def _gpu(*shape, dtype=torch.float32, cls=Gpu):
    return torch.zeros(*shape, dtype=dtype).as_subclass(cls)


def test_residual_norm_binding_refuses(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = _gpu(6, 64)
    with pytest.raises(ValueError, match="whole samples"):
        B.residual_norm_fwd(x, x, x, x, positions=4)
    with pytest.raises(ValueError, match="gate must be 3 x 64"):
        B.residual_norm_fwd(x, x, x, x, positions=2, gate=_gpu(6, 64))
    with pytest.raises(TypeError, match="u must be"):
        B.residual_norm_fwd(x, x, x, _gpu(6, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="post_stats has"):
        B.residual_norm_fwd(x, x, x, x, post_stats=_gpu(6))
    with pytest.raises(ValueError, match="GPU"):
        B.residual_norm_fwd(x, torch.zeros(6, 64), x, x)
    with pytest.raises(ValueError, match="dh must be"):
        B.residual_norm_bwd(x, x, x, x, x, _gpu(6, 32))
    # tensors of another device than the current one, whose stream the call would enter
    with pytest.raises(ValueError, match="current device is cuda:0"):
        B.residual_norm_fwd(x, _gpu(6, 64, cls=Other), x, x, stream=0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        B.residual_norm_bwd(x, x, x, x, x, x, post_stats=_gpu(6, 2), pre_stats=_gpu(6, 2, cls=Other), stream=0)


def test_stacks_refuse_rows_that_would_be_broadcast():
    """The gradient of x that backward returns has a row for every node, so x must have them, too."""
    from types import SimpleNamespace
    from quantized_halo_aggregation_amd.training import GatedNormStack, ResidualStack
    held = torch.zeros(6, 8)
    for stack in (GatedNormStack, ResidualStack):
        for shape in ((8,), (1, 8), (6, 1), (), (6, 8, 1), (5, 8)):
            with pytest.raises(ValueError, match="6 x 8"):
                stack.forward(SimpleNamespace(gp=None, X=[held], layers=1), torch.ones(shape))
    assert not held.any()


def _coef(k=B.NS_COEFFICIENTS, steps=5):
    return B._ns_coefficients(k, steps)


def _table(rows):
    import numpy as np
    return np.array(rows, dtype=np.int64).reshape(len(rows), -1)


GOOD_NS = (200, 300, FAKE, 300, FAKE, 300)


def _ns(rows=(GOOD_NS,), n=None, t=B.F32, o=B.F32, steps=5, k=None, eps=1e-7, ws=FAKE, wsb=1 << 40):
    table = _table(rows) if rows else None
    k = _coef(steps=5) if k is None else k
    return B._newton_schulz(None if table is None else table.ctypes.data, len(rows) if n is None else n, t, o, steps,
                            k if isinstance(k, int) else k.ctypes.data, eps, ws, wsb, None)


GOOD_MUON = (200, 300, FAKE, FAKE, FAKE, FAKE, 1.0)


def _muon(rows=(GOOD_MUON,), n=None, gt=B.F32, ct=B.F32, lr=0.02, beta=0.95, wd=0.1, gs=1.0, steps=5, k=None, eps=1e-7,
          ws=FAKE, wsb=1 << 40):
    import numpy as np
    table = np.zeros((max(len(rows), 1), 7), np.int64)
    for i, r in enumerate(rows):
        table[i, :6] = r[:6]
        table.view(np.float64)[i, 6] = r[6]
    k = _coef(steps=5) if k is None else k
    return B._muon_step(table.ctypes.data if rows else None, len(rows) if n is None else n, gt, ct, lr, beta, 1, wd, gs, steps,
                        k if isinstance(k, int) else k.ctypes.data, eps, ws, wsb, None)


STEPS = [dict(n=-1), dict(steps=0), dict(steps=17), dict(steps=-1), dict(k=0), dict(eps=-1.0), dict(eps=NAN), dict(rows=(), n=1),
         dict(k=_coef((40, 0, 0))), dict(k=_coef((4, -7, 4))), dict(k=_coef((NAN, 0, 0))), dict(k=_coef((1, float("inf"), 0))),
         dict(k=_coef((0, 0, -70))),
         # 1.99 after the first step, 6.9 - 37.8 + 64 after the second
         dict(k=_coef([(8.2872, -23.5959, 17.3004)] + [(3.4445, -4.7750, 2.0315)] * 4)), dict(k=_coef((0, 240, -240))), dict(ws=FAKE + 8)]


@pytest.mark.parametrize("bad", STEPS + [
    dict(t=3), dict(o=-1), dict(rows=((-1, 300, FAKE, 300, FAKE, 300),)), dict(rows=((200, 300, 0, 300, FAKE, 300),)),
    dict(rows=((200, 300, FAKE, 300, 0, 300),)), dict(rows=((200, 300, FAKE, 299, FAKE, 300),)),
    dict(rows=((200, 300, FAKE, 300, FAKE, 0),)), dict(rows=((200, 300, FAKE + 2, 300, FAKE, 300),)),
    dict(rows=((200, 300, FAKE + 1, 300, FAKE, 300),), t=B.BF16), dict(rows=((200, 300, FAKE, 300, FAKE + 1, 300),), o=B.F16),
    dict(rows=(GOOD_NS, (4, 4, 0, 4, FAKE, 4)))])
def test_newton_schulz_refuses(bad):
    assert _ns(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


@pytest.mark.parametrize("bad", STEPS + [
    dict(gt=3), dict(ct=-1), dict(lr=-1.0), dict(lr=NAN), dict(lr=1e300), dict(beta=1.0), dict(beta=-0.1), dict(beta=NAN),
    dict(wd=-1.0), dict(wd=float("inf")), dict(gs=NAN), dict(gs=1e300),
    dict(rows=((200, -3, FAKE, FAKE, 0, FAKE, 1.0),)), dict(rows=((200, 300, 0, FAKE, 0, FAKE, 1.0),)),
    dict(rows=((200, 300, FAKE, 0, 0, FAKE, 1.0),)), dict(rows=((200, 300, FAKE, FAKE, 0, 0, 1.0),)),
    dict(rows=((200, 300, FAKE + 2, FAKE, 0, FAKE, 1.0),)), dict(rows=((200, 300, FAKE, FAKE + 2, 0, FAKE, 1.0),)),
    dict(rows=((200, 300, FAKE, FAKE, 0, FAKE + 2, 1.0),)), dict(rows=((200, 300, FAKE, FAKE, FAKE + 1, FAKE, 1.0),), ct=B.BF16),
    dict(rows=((200, 300, FAKE, FAKE, 0, FAKE, -1.0),)), dict(rows=((200, 300, FAKE, FAKE, 0, FAKE, NAN),)),
    dict(rows=(GOOD_MUON, (4, 4, FAKE, FAKE, 0, 0, 1.0)))])
def test_muon_step_refuses(bad):
    assert _muon(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


def test_newton_schulz_limits_and_workspace():
    far = ((1 << 17, 4, FAKE, 4, FAKE, 4),)
    assert _ns(rows=far) == B.QHA_ERR_UNSUPPORTED
    assert _muon(rows=((4, 1 << 17, FAKE, FAKE, 0, FAKE, 1.0),)) == B.QHA_ERR_UNSUPPORTED
    assert _ns(ws=None) == B.QHA_ERR_WORKSPACE and _muon(ws=None) == B.QHA_ERR_WORKSPACE
    need = B.newton_schulz_workspace([(200, 300)])
    assert need > 0 and _ns(wsb=need - 1) == B.QHA_ERR_WORKSPACE
    # a matrix and its transpose need the same but for the sums of squares of their pieces
    assert abs(need - B.newton_schulz_workspace([(300, 200)])) <= 8 * 64
    assert B.newton_schulz_workspace([(128, 128), (1, 5), (0, 700), (700, 0)]) == 0      # on chip, or nothing to do
    assert B.newton_schulz_workspace([(128, 129)]) > 0
    assert B.newton_schulz_workspace([(200, 300), (1 << 17, 4)]) == 0
    for steps in (0, 17):
        assert B.newton_schulz_workspace([(200, 300)], steps) == 0
    # a long list is worked off in batches that share the space
    assert B.newton_schulz_workspace([(1024, 1024)] * 400) < 50 * B.newton_schulz_workspace([(1024, 1024)])
    assert _ns(rows=()) == B.QHA_OK and _muon(rows=()) == B.QHA_OK
    assert _ns(rows=((0, 5, 0, 0, 0, 0), (5, 0, 0, 0, 0, 0)), ws=None) == B.QHA_OK
    assert _muon(rows=((0, 5, 0, 0, 0, 0, 1.0),), ws=None) == B.QHA_OK


def test_coefficients_that_stay_in_range_are_taken():
    for k, steps in ((B.NS_COEFFICIENTS, 16), ((1.5, -0.5, 0.0), 16), ((15 / 8, -10 / 8, 3 / 8), 9), ((0, 0, 0), 1), ((3.8, 0, 0), 1),
                     ([(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448)], 2)):
        assert B._newton_schulz(None, 0, B.F32, B.F32, steps, B._ns_coefficients(k, steps).ctypes.data, 0.0, None, 0, None) == B.QHA_OK
    # |5 s - 20 s^3 + 16 s^5| <= 1 on [0, 1], but its slope at 1 is 25: a rounding there grows 25-fold a step
    five_fold = lambda n: B._newton_schulz(None, 0, B.F32, B.F32, n, B._ns_coefficients((5, -20, 16), n).ctypes.data, 0.0, None, 0, None)
    assert five_fold(2) == B.QHA_OK and five_fold(5) == B.QHA_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="coefficients"):
        B._ns_coefficients([(1, 2, 3)] * 4, 5)
    with pytest.raises(ValueError, match="coefficients"):
        B._ns_coefficients((1, 2), 5)


def test_coefficients_of_any_size_are_checked():
    """The bounds are formed in float64, whose squares and sums of the largest coefficients are infinite, and the steps in float32,
    which ends at 3.4e38."""
    def status(k, steps=1):
        return B._newton_schulz(None, 0, B.F32, B.F32, steps, B._ns_coefficients(k, steps).ctypes.data, 0.0, None, 0, None)
    big = 1.7e308
    # at s^2 = 1/2 the first is 1 - 2.5e307; the others pass at the end, or inside [0, 1]
    for k in ((1, -1e308, 1e308), (1, -big, big), (0, big, -big), (1, 0, big), (big, -big, 0), (-big, big, 1), (1, -1e154, 1e154),
              (1, 1e300, -1e300), (0, 0, -big)):
        assert status(k) == B.QHA_ERR_INVALID_ARG, k
        assert status([B.NS_COEFFICIENTS, k], 2) == B.QHA_ERR_INVALID_ARG, k
    # singular values of up to 1e-3, 1e-150 and 0 would bear these, float32 does not
    for first, k in ((1e-3, (1, -1e300, 0)), (1e-150, (1, 1e299, 0)), (1e-150, (1, 0, 1e300)), (0, (1, 1e300, -1e300)), (0, (0, 0, 1e39))):
        assert status([(first, 0, 0), k], 2) == B.QHA_ERR_INVALID_ARG, k
    # and these it does: 3 - 3 + 3 at s = 1e-3
    assert status([(1e-3, 0, 0), (3, -3e6, 3e12)], 2) == B.QHA_OK
    assert status([(1e-3, 0, 0), (3, -3e6, 70e12)], 2) == B.QHA_ERR_INVALID_ARG


def test_newton_schulz_and_muon_binding_refuse(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = _gpu(4, 6)
    with pytest.raises(ValueError, match="2 results for 1"):
        B.newton_schulz([x], [x, x])
    with pytest.raises(ValueError, match="matrix"):
        B.newton_schulz([_gpu(4)], [x])
    with pytest.raises(ValueError, match="4 x 6"):
        B.newton_schulz([x], [_gpu(6, 4)])
    with pytest.raises(TypeError, match="float32"):
        B.newton_schulz([x, _gpu(4, 6, dtype=torch.bfloat16)], [x, x])
    with pytest.raises(ValueError, match="two of the results"):
        B.newton_schulz([x, _gpu(4, 6)], [x, x])
    with pytest.raises(ValueError, match="GPU"):
        B.newton_schulz([torch.zeros(4, 6)], [x])
    with pytest.raises(ValueError, match="current device"):
        B.newton_schulz([x], [_gpu(4, 6, cls=Other)], stream=0)
    with pytest.raises(ValueError, match="passes 60|pass 3.8"):
        B.newton_schulz([x], [x], coefficients=(40, 0, 0), stream=0)
    with pytest.raises(ValueError, match="coefficients"):
        B.newton_schulz([x], [x], coefficients=(1, 2))
    with pytest.raises(TypeError, match="float32"):
        B.Muon([_gpu(4, 6, dtype=torch.float16)])
    with pytest.raises(ValueError, match="matrix"):
        B.Muon([_gpu(24)])
    with pytest.raises(ValueError, match="contiguous"):
        B.Muon([_gpu(6, 4).T])
    with pytest.raises(ValueError, match="scale"):
        B.Muon([x], scale="spectrum")
    with pytest.raises(ValueError, match="momenta"):
        B.Muon([x], momenta=[])
    with pytest.raises(ValueError, match=r"m\[0\] must be"):
        B.Muon([x], momenta=[_gpu(6, 4)])
    with pytest.raises(ValueError, match=r"copies\[0\] must be"):
        B.Muon([x], copies=[_gpu(24)])
    for again in ({"params": [x, x]}, {"params": [x], "momenta": [x]}, {"params": [x], "copies": [x]}):
        with pytest.raises(ValueError, match="same memory"):
            B.Muon(**again)
    B.Muon([_gpu(0, 6), _gpu(0, 6)])
    opt = B.Muon([x])
    with pytest.raises(ValueError, match="2 gradients for 1"):
        opt.step([x, x], 0.1)
    with pytest.raises(ValueError, match=r"grads\[0\] must be"):
        opt.step([_gpu(24)], 0.1)
    with pytest.raises(TypeError, match="float32|float16"):
        opt.step([_gpu(4, 6, dtype=torch.float64)], 0.1)
    with pytest.raises(ValueError, match="current device"):
        opt.step([_gpu(4, 6, cls=Other)], 0.1, stream=0)
    B.Muon([]).step([], 0.1)


@pytest.fixture
def muon_calls(monkeypatch):
    """The (table, gradients' type, copies' type) of every qha_muon_step, recorded in its place."""
    import numpy as np
    calls = []

    def record(table, n, grad_type, copy_type, *rest):
        import ctypes
        rows = np.ctypeslib.as_array((ctypes.c_int64 * (7 * n)).from_address(table)).reshape(n, 7).copy()
        calls.append((rows, grad_type, copy_type))
        return B.QHA_OK
    monkeypatch.setattr(B, "_muon_step", record)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return calls


def test_muon_without_its_copies_writes_none(muon_calls):
    """Copies that were given up are not written any more, and are again when they come back."""
    copies = [_gpu(4, 6, dtype=torch.bfloat16), _gpu(9, 3, dtype=torch.bfloat16)]
    opt = B.Muon([_gpu(4, 6), _gpu(9, 3)], copies=copies)
    grads = [_gpu(4, 6), _gpu(9, 3)]
    for now in (copies, None, copies, None):
        opt.copies = now
        opt.step(grads, 0.1, stream=0)
        rows, _, copy_type = muon_calls[-1]
        assert rows[:, 4].tolist() == ([0, 0] if now is None else [c.data_ptr() for c in copies])
        assert copy_type == (B.F32 if now is None else B.BF16)


def test_muon_checks_what_stands_at_a_known_address(muon_calls):
    """Views of the memory that was there at the last step, with another type, shape or order of their elements."""
    copies = [_gpu(4, 4, dtype=torch.bfloat16)]
    opt = B.Muon([_gpu(4, 4)], copies=copies)
    step = lambda: opt.step([_gpu(4, 4)], 0.1, stream=0)
    step()
    assert muon_calls[-1][2] == B.BF16
    opt.copies = [copies[0].view(torch.float16)]
    step()
    assert muon_calls[-1][2] == B.F16
    calls = len(muon_calls)
    opt.copies = [copies[0].view(torch.int16)]
    with pytest.raises(TypeError):
        step()
    opt.copies = copies
    for name in ("params", "m", "copies"):
        own = getattr(opt, name)
        for bad, what in ((own[0].t(), "contiguous"), (own[0].view(2, 8), "must be"), (own[0][:3], "must be"),
                          (own[0].as_strided((4, 4), (2, 1)), "contiguous")):
            assert bad.data_ptr() == own[0].data_ptr()
            setattr(opt, name, [bad])
            with pytest.raises(ValueError, match=what):
                step()
        setattr(opt, name, own)
    # the same object, turned in its place
    opt.params[0].t_()
    with pytest.raises(ValueError, match="contiguous"):
        step()
    assert len(muon_calls) == calls
    opt.params[0].t_()
    step()
    assert len(muon_calls) == calls + 1


def test_results_over_inputs_of_others_are_refused(monkeypatch):
    """Matrices of one launch are read and written at once, so a result may lie over its own input alone, place by place;
    gradients are read again after the momenta were written."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    done = []
    monkeypatch.setattr(B, "_newton_schulz", lambda *args: done.append(args) or B.QHA_OK)
    monkeypatch.setattr(B, "_muon_step", lambda *args: done.append(args) or B.QHA_OK)
    x, y, z = _gpu(4, 4), _gpu(4, 4), _gpu(4, 4)
    buf = _gpu(8, 8)
    for xs, outs in (([x, y], [y, x]), ([x, y], [z, x]), ([x, x], [x, z]), ([buf[:4, :4]], [buf.view(-1)[:16].view(4, 4)]),
                     ([x], [x.view(torch.float16).view(-1)[:16].view(4, 4)])):
        with pytest.raises(ValueError, match="another matrix|in place"):
            B.newton_schulz(xs, outs, stream=0)
    opt = B.Muon([x, y], copies=[z, _gpu(4, 4)])
    for grads in ([opt.m[1], z], [x, _gpu(4, 4)], [opt.copies[1], _gpu(4, 4)]):
        with pytest.raises(ValueError, match="gradient"):
            opt.step(grads, 0.1, stream=0)
    assert not done
    empty = _gpu(0, 4)
    B.newton_schulz([x, x, buf[:4, :4], empty, empty], [y, z, buf[:4, :4], empty, _gpu(0, 4)], stream=0)
    opt.step([_gpu(4, 4)] * 2, 0.1, stream=0)              # gradients that are read alone may be the same
    B.Muon([empty]).step([empty], 0.1, stream=0)
    assert len(done) == 3


def test_muon_table_follows_the_tensors(monkeypatch):
    """The addresses that reach the library, after parameters and momenta were replaced, without a GPU."""
    import numpy as np
    seen = []

    def fake(table, n, *rest):
        import ctypes
        seen.append(np.ctypeslib.as_array((ctypes.c_int64 * (7 * n)).from_address(table)).reshape(n, 7).copy())
        return B.QHA_OK
    monkeypatch.setattr(B, "_muon_step", fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    params = [_gpu(4, 6), _gpu(9, 3)]
    copies = [_gpu(4, 6, dtype=torch.bfloat16), _gpu(9, 3, dtype=torch.bfloat16)]
    grads = [_gpu(4, 6), _gpu(9, 3)]
    opt = B.Muon(params, scale="spectral", copies=copies)

    def expect():
        opt.step(grads, 0.1, stream=0)
        t = seen[-1]
        assert t[:, :2].tolist() == [[4, 6], [9, 3]]
        assert t[:, 2].tolist() == [p.data_ptr() for p in opt.params]
        assert t[:, 3].tolist() == [g.data_ptr() for g in grads]
        assert t[:, 4].tolist() == [c.data_ptr() for c in opt.copies]
        assert t[:, 5].tolist() == [m.data_ptr() for m in opt.m]
        assert t.view(np.float64)[:, 6].tolist() == [1.0, 3 ** 0.5]
    expect()
    opt.params[1] = _gpu(9, 3)
    expect()
    opt.m[0] = _gpu(4, 6)
    expect()
    grads[0] = _gpu(4, 6)
    opt.copies[1] = _gpu(9, 3, dtype=torch.bfloat16)
    expect()
    opt.m.pop()
    with pytest.raises(ValueError, match="momenta"):
        opt.step(grads, 0.1, stream=0)
    assert B.Muon(params, scale="rms")._table.view(np.float64)[0, 6] == 0.2 * 6 ** 0.5
    assert B.Muon(params, scale=0.5)._table.view(np.float64)[0, 6] == 0.5
