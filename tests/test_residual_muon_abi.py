"""Refusals of the residual norm's entry points and of their binding, without a GPU.

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
