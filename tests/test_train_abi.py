"""Refusals of the training operators' entry points and of their binding, without a GPU.

Argument-error cases pass fake (never dereferenced) device addresses: the checks must fire first.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from quantized_halo_aggregation_amd import binding as B

FAKE = 0x10000
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _adam(tensors=((10, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE),), n=None, bits=32, gt=B.F32, ct=B.F32, lr=1e-3, b1=0.9,
          b2=0.999, eps=1e-8, wd=0.01, scale=1.0, step=1):
    table = np.array(tensors, dtype=np.int64).reshape(-1, 8)
    return B._adamw_step(table.ctypes.data if table.size else None, len(table) if n is None else n, bits, gt, ct, lr, b1,
                         b2, eps, wd, scale, step, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(bits=16), dict(gt=3), dict(ct=-1), dict(lr=-1.0), dict(lr=float("nan")), dict(eps=-1e-9),
    dict(wd=float("inf")), dict(scale=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(b2=float("nan")), dict(step=0),
    dict(tensors=(), n=1),
    dict(tensors=((-1, FAKE, FAKE, 0, FAKE, FAKE, 0, 0),)),
    dict(tensors=((1 << 41, FAKE, FAKE, 0, FAKE, FAKE, 0, 0),)),
    dict(tensors=((10, 0, FAKE, 0, FAKE, FAKE, 0, 0),)),
    dict(tensors=((10, FAKE, 0, 0, FAKE, FAKE, 0, 0),)),
    dict(tensors=((10, FAKE, FAKE, 0, 0, FAKE, 0, 0),)),
    dict(tensors=((10, FAKE, FAKE, 0, FAKE, 0, 0, 0),)),
    dict(tensors=((10, FAKE, FAKE, 0, FAKE, FAKE, 0, FAKE),), bits=8),
    dict(tensors=((10, FAKE, FAKE, 0, FAKE, FAKE, FAKE, 0),), bits=8),
    dict(tensors=((10, FAKE + 2, FAKE, 0, FAKE, FAKE, 0, 0),)),
    dict(tensors=((10, FAKE, FAKE + 2, 0, FAKE, FAKE, 0, 0),)),
    dict(tensors=((10, FAKE, FAKE + 1, 0, FAKE, FAKE, 0, 0),), gt=B.BF16),
    dict(tensors=((10, FAKE, FAKE, FAKE + 1, FAKE, FAKE, 0, 0),), ct=B.F16),
    dict(tensors=((10, FAKE, FAKE, 0, FAKE + 2, FAKE, 0, 0),)),
    dict(tensors=((10, FAKE, FAKE, 0, FAKE, FAKE, FAKE + 2, FAKE),), bits=8),
    # a bad tensor after a good one
    dict(tensors=((10, FAKE, FAKE, 0, FAKE, FAKE, 0, 0), (10, FAKE, FAKE, 0, FAKE, 0, 0, 0))),
])
def test_adamw_step_refuses(bad):
    assert _adam(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


def test_adamw_step_without_elements_is_ok():
    assert _adam(tensors=()) == B.QHA_OK
    assert _adam(tensors=((0, 0, 0, 0, 0, 0, 0, 0),) * 60) == B.QHA_OK


def test_adamw_values_refuses():
    v = B._adamw_values
    assert v(FAKE, FAKE, FAKE, None, None, None, -1, None) == B.QHA_ERR_INVALID_ARG
    assert v(FAKE, None, FAKE, None, None, None, 5, None) == B.QHA_ERR_INVALID_ARG
    assert v(None, None, None, FAKE, FAKE, None, 5, None) == B.QHA_ERR_INVALID_ARG
    assert v(FAKE, FAKE, FAKE + 2, None, None, None, 5, None) == B.QHA_ERR_INVALID_ARG
    assert v(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None) == B.QHA_OK
    assert v(None, None, None, None, None, None, 5, None) == B.QHA_OK


def test_adamw_binding_refuses():
    with pytest.raises(ValueError, match="8 or 32"):
        B.AdamW([], bits=16)
    with pytest.raises(TypeError, match="float32"):
        B.AdamW([torch.zeros(4, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="GPU"):
        B.AdamW([torch.zeros(4)])
    with pytest.raises(TypeError, match="tensor"):
        B.AdamW([np.zeros(4, np.float32)])
    with pytest.raises(ValueError, match="copies"):
        B.AdamW([], copies=[torch.zeros(4)])


def _norm_fwd(n=10, p=300, c=64, g=4, t=B.F32, x=FAKE, ldx=64, w=FAKE, b=FAKE, eps=1e-5, act=0, y=FAKE, ldy=64, mean=FAKE,
              rstd=FAKE, ws=FAKE, wsb=1 << 30):
    return B._group_norm_fwd(n, p, c, g, t, x, ldx, w, b, eps, act, y, ldy, mean, rstd, ws, wsb, None)


def _norm_bwd(n=10, p=300, c=64, g=4, t=B.F32, dy=FAKE, lddy=64, x=FAKE, ldx=64, mean=FAKE, rstd=FAKE, w=FAKE, b=FAKE,
              act=0, dx=FAKE, lddx=64, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30):
    return B._group_norm_bwd(n, p, c, g, t, dy, lddy, x, ldx, mean, rstd, w, b, act, dx, lddx, dw, db, ws, wsb, None)


SHARED = [dict(n=-1), dict(p=0), dict(n=1 << 20, p=1 << 20), dict(c=0), dict(c=66), dict(c=60, t=B.BF16), dict(g=0), dict(g=5),
          dict(t=3), dict(act=4), dict(act=-1), dict(w=FAKE + 4), dict(b=FAKE + 8), dict(x=None), dict(x=FAKE + 4),
          dict(ldx=60), dict(ldx=66), dict(ldx=68, t=B.F16), dict(ws=FAKE + 8)]


@pytest.mark.parametrize("bad", SHARED + [dict(y=None), dict(ldy=32), dict(y=FAKE + 2), dict(eps=-1.0),
                                          dict(eps=float("inf")), dict(mean=None), dict(rstd=None), dict(mean=FAKE + 2)])
def test_group_norm_fwd_refuses(bad):
    assert _norm_fwd(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


@pytest.mark.parametrize("bad", SHARED + [dict(dy=None), dict(lddy=0), dict(dx=None), dict(lddx=62), dict(mean=None),
                                          dict(rstd=None), dict(dw=None), dict(db=None), dict(dw=FAKE + 2)])
def test_group_norm_bwd_refuses(bad):
    assert _norm_bwd(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


def test_group_norm_limits_and_workspace():
    wide = dict(c=8448, ldx=8448, g=1)
    assert _norm_fwd(ldy=8448, **wide) == B.QHA_ERR_UNSUPPORTED
    assert _norm_bwd(lddy=8448, lddx=8448, **wide) == B.QHA_ERR_UNSUPPORTED
    assert B.group_norm_workspace(3000, 300, 64, 4, backward=True) > 0
    assert B.group_norm_workspace(30, 3, 64, 4) == 0        # samples held in registers need none forward
    assert B.group_norm_workspace(30, 3, 64, 4, backward=True) > 0
    assert _norm_bwd(ws=None) == B.QHA_ERR_WORKSPACE
    assert _norm_bwd(wsb=15) == B.QHA_ERR_WORKSPACE
    assert _norm_fwd(ws=None, wsb=0) == B.QHA_ERR_WORKSPACE
    assert _norm_fwd(n=0, x=None, y=None) == B.QHA_OK
    assert _norm_bwd(n=0, dw=None, db=None, x=None) == B.QHA_OK
    assert B.group_norm_workspace(0, 1, 64, 4) == 0


def test_group_norm_binding_refuses():
    x = torch.zeros(6, 16)
    with pytest.raises(ValueError, match="GPU"):
        B.group_norm_fwd(x, x, 2)
    with pytest.raises(ValueError, match="whole samples"):
        B.group_norm_fwd(x, x, 2, positions=4)


def _gated_fwd(m=10, n=64, k=32, t=B.F32, a=FAKE, lda=32, wg=FAKE, ldwg=32, wu=FAKE, ldwu=32, act=2, h=FAKE, ldh=64,
               gate=FAKE, ldg=64, up=FAKE, ldu=64, ws=FAKE, wsb=1 << 30):
    return B._gated_project(m, n, k, t, a, lda, wg, ldwg, wu, ldwu, act, h, ldh, gate, ldg, up, ldu, ws, wsb, None)


def _gated_bwd(m=10, n=64, k=32, t=B.F32, dh=FAKE, lddh=64, gate=FAKE, ldg=64, up=FAKE, ldu=64, a=FAKE, lda=32, wg=FAKE,
               ldwg=32, wu=FAKE, ldwu=32, act=2, da=FAKE, ldda=32, dwg=FAKE, lddwg=32, dwu=FAKE, lddwu=32, ws=FAKE,
               wsb=1 << 30):
    return B._gated_backward(m, n, k, t, dh, lddh, gate, ldg, up, ldu, a, lda, wg, ldwg, wu, ldwu, act, da, ldda, dwg,
                             lddwg, dwu, lddwu, ws, wsb, None)


GATED = [dict(m=-1), dict(n=-8), dict(k=-8), dict(n=62), dict(k=30), dict(k=36, t=B.BF16, lda=40, ldwg=40, ldwu=40),
         dict(n=1 << 17), dict(t=5), dict(act=7), dict(a=None), dict(a=FAKE + 4), dict(lda=28), dict(lda=34), dict(wg=None),
         dict(ldwg=16), dict(wu=FAKE + 8), dict(ldwu=33), dict(ldg=60), dict(up=FAKE + 2), dict(ldu=0), dict(gate=None),
         dict(up=None), dict(m=1000, ws=FAKE + 8)]


@pytest.mark.parametrize("bad", GATED + [dict(h=None), dict(ldh=63), dict(h=FAKE + 8), dict(k=0)])
def test_gated_project_refuses(bad):
    assert _gated_fwd(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


@pytest.mark.parametrize("bad", GATED + [dict(dh=None), dict(lddh=32), dict(da=FAKE + 4), dict(ldda=31), dict(dwg=None),
                                         dict(lddwg=30), dict(dwu=None), dict(dwu=FAKE + 4), dict(lddwu=28), dict(n=0),
                                         dict(k=0)])
def test_gated_backward_refuses(bad):
    assert _gated_bwd(**bad) == B.QHA_ERR_INVALID_ARG
    assert B._last_error()


def test_gated_limits_and_workspace():
    assert B.gated_project_workspace(torch.bfloat16, 1000, 64, 32) == 0
    assert B.gated_project_workspace(torch.float32, 1000, 64, 32) > 0
    assert B.gated_project_workspace(torch.float32, 10, 64, 32) == 0        # few rows need none
    assert _gated_fwd(m=1000, ws=None, wsb=0) == B.QHA_ERR_WORKSPACE
    assert _gated_bwd(wsb=100) == B.QHA_ERR_WORKSPACE
    assert _gated_fwd(m=0, a=None, h=None, ws=None, wsb=0) == B.QHA_OK
    assert _gated_fwd(m=1 << 30, n=1 << 12, ldh=1 << 12, ldg=1 << 12, ldu=1 << 12) == B.QHA_ERR_UNSUPPORTED
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        B.gated_project_workspace(torch.float64, 1, 8, 8)


def test_gated_binding_refuses():
    a, w, h = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        B.gated_project(a, w, w, h)


def test_group_norm_workspace_of_narrow_rows():
    """Widths below a 16-bit vector: four float32 channels are legal, one to three and five to seven are not, and twelve suit
    float32 alone.  In a process of its own, because a division by zero on the host would end this one."""
    code = ("from quantized_halo_aggregation_amd import binding as B\n"
            "for c in list(range(1, 9)) + [12]:\n"
            "    for rows, positions in ((300, 1), (300, 100), (6000, 3000)):\n"
            "        print(c, positions, *(B.group_norm_workspace(rows, positions, c, 1, b) for b in (False, True)))\n")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert res.returncode == 0, (res.returncode, res.stderr[-500:])
    got = {tuple(map(int, line.split()[:2])): tuple(map(int, line.split()[2:])) for line in res.stdout.splitlines()}
    assert len(got) == 27
    for (c, positions), (fwd, bwd) in got.items():
        if c % 4:
            assert (fwd, bwd) == (0, 0), c
            continue
        assert bwd >= 2 * c * 4 and (fwd > 0 or positions < 3000), (c, positions, fwd, bwd)
        if c % 8:        # float32 is the only type of these: the query gives exactly what the calls ask for
            shape = dict(n={1: 300, 100: 3, 3000: 2}[positions], p=positions, c=c, g=1)
            assert _norm_bwd(ldx=c, lddy=c, lddx=c, wsb=bwd - 1, **shape) == B.QHA_ERR_WORKSPACE
            if fwd:
                assert _norm_fwd(ldx=c, ldy=c, wsb=fwd - 1, **shape) == B.QHA_ERR_WORKSPACE


@pytest.fixture
def adamw_calls(monkeypatch):
    """AdamW over host tensors, with the tables that would reach qha_adamw_step recorded in its place."""
    tables = []

    def record(table, n, *rest):
        import ctypes
        tables.append(np.ctypeslib.as_array((ctypes.c_int64 * (8 * n)).from_address(table)).reshape(n, 8).copy())
        return B.QHA_OK
    check = B._flat

    def on_host(t, name, n=None, dtype=None):
        class Gpu(torch.Tensor):
            is_cuda = True
        return check(t.as_subclass(Gpu) if isinstance(t, torch.Tensor) else t, name, n, dtype)
    monkeypatch.setattr(B, "_adamw_step", record)
    monkeypatch.setattr(B, "_flat", on_host)
    return tables


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_writes_where_its_tensors_are_now(adamw_calls, bits):
    """Parameters whose .data was replaced, and moments, scales and copies that were assigned on resume."""
    params = [torch.zeros(300), torch.zeros(5)]
    opt = B.AdamW(params, bits=bits, copies=[torch.zeros(300, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.bfloat16)])
    grads = [torch.zeros(300), torch.zeros(5)]

    def expect():
        opt.step(grads, 1e-3, stream=0)
        t, e = adamw_calls[-1], 4 if bits == 32 else 1
        assert t[:, 0].tolist() == [300, 5]
        assert t[:, 1].tolist() == [p.data_ptr() for p in params]
        assert t[:, 2].tolist() == [g.data_ptr() for g in grads]
        assert t[:, 3].tolist() == [c.data_ptr() for c in opt.copies]
        assert t[:, 4].tolist() == [opt.m.data_ptr() + s * e for s in opt.starts]
        assert t[:, 5].tolist() == [opt.v.data_ptr() + s * e for s in opt.starts]
        if bits == 8:
            assert t[:, 6].tolist() == [opt.m_scale.data_ptr() + s // 256 * 4 for s in opt.starts]
            assert t[:, 7].tolist() == [opt.v_scale.data_ptr() + s // 256 * 4 for s in opt.starts]
    expect()
    params[1].data = torch.ones(5)
    expect()
    for name in ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
        setattr(opt, name, getattr(opt, name).clone())
        expect()
    opt.copies[0] = opt.copies[0].clone()
    expect()
    opt.m.data = opt.m.clone()
    expect()
    # what does not fit is refused, and goes nowhere
    calls, t = len(adamw_calls), opt.t
    for name, bad in (("m", opt.m[:-1].clone()), ("v", opt.v.double()), ("m", opt.m.repeat(2)[::2])):
        good = getattr(opt, name)
        setattr(opt, name, bad)
        with pytest.raises((ValueError, TypeError), match=name):
            opt.step(grads, 1e-3, stream=0)
        setattr(opt, name, good)
    params[0].data = torch.zeros(299)
    with pytest.raises(ValueError, match="params"):
        opt.step(grads, 1e-3, stream=0)
    assert len(adamw_calls) == calls and opt.t == t
    params[0].data = torch.zeros(300)
    expect()
    with pytest.raises(AttributeError):
        opt.bits = 40 - bits


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_without_its_copies_writes_none(adamw_calls, bits):
    """Copies that were given up are not written any more, and are again when they come back."""
    copies = [torch.zeros(300, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.bfloat16)]
    opt = B.AdamW([torch.zeros(300), torch.zeros(5)], bits=bits, copies=copies)
    for now in (copies, None, copies, None):
        opt.copies = now
        opt.step([torch.zeros(300), torch.zeros(5)], 1e-3, stream=0)
        assert adamw_calls[-1][:, 3].tolist() == ([0, 0] if now is None else [c.data_ptr() for c in copies])


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_checks_what_stands_at_a_known_address(adamw_calls, bits, monkeypatch):
    """Views of the memory that was there at the last step, with another type, size or order of their elements."""
    types, record = [], B._adamw_step

    def with_type(table, n, state_bits, grad_type, copy_type, *rest):
        types.append(copy_type)
        return record(table, n, state_bits, grad_type, copy_type, *rest)
    monkeypatch.setattr(B, "_adamw_step", with_type)
    copies = [torch.zeros(16, 16, dtype=torch.bfloat16)]
    opt = B.AdamW([torch.zeros(16, 16)], bits=bits, copies=copies)
    step = lambda: opt.step([torch.zeros(16, 16)], 1e-3, stream=0)
    step()
    opt.copies = [copies[0].view(torch.float16)]
    step()
    assert types == [B.BF16, B.F16]
    opt.copies = copies
    for name in ("params", "copies"):
        own = getattr(opt, name)
        for bad, what in ((own[0].t(), "contiguous"), (own[0][:3], "elements")):
            assert bad.data_ptr() == own[0].data_ptr()
            setattr(opt, name, [bad])
            with pytest.raises(ValueError, match=what):
                step()
        setattr(opt, name, own)
    for name in ("m", "v"):
        own = getattr(opt, name)
        for bad in (own.view(torch.float16 if bits == 32 else torch.bool), own[:128]):
            setattr(opt, name, bad)
            with pytest.raises((ValueError, TypeError), match=name):
                step()
        setattr(opt, name, own)
    opt.params[0].t_()                   # the same object, turned in its place
    with pytest.raises(ValueError, match="contiguous"):
        step()
    assert len(types) == 2
    opt.params[0].t_()
    step()
    assert len(types) == 3


def test_the_stride_of_a_single_row_does_not_matter():
    """One row of a buffer with odd rows (one token, one node) has no next row: its leading dimension is its width."""
    class Gpu(torch.Tensor):
        is_cuda = True
    buf = torch.zeros(3, 67)
    for view in (buf[:1, :64], buf[1:2, 1:65], torch.zeros(64).expand(1, 64)):
        p, ld = B._matrix(view.as_subclass(Gpu), "a", torch.float32, 1, 64)
        assert (p, ld) == (view.data_ptr(), 64)
        assert _norm_fwd(n=1, p=1, ldx=ld, ldy=ld, mean=None, rstd=None, x=FAKE + 4, ws=None, wsb=0) == B.QHA_ERR_INVALID_ARG
        assert b"aligned" in B._last_error()
    assert B._matrix(buf[:2, :64].as_subclass(Gpu), "a", torch.float32, 2, 64)[1] == 67
