"""What gl_rmsnorm and gl_rmsnorm_bwd refuse, before any CUDA call (no GPU)."""
import pytest
import torch

from grouped_gemm_splits_b200 import gl

BF, U8 = torch.bfloat16, torch.uint8


def _c(x=16, r=None, g=16, eps=1e-5, rows=4, cols=128, sum=None, y=32, rstd=None, codes=None, scales=None, layout=0):
    return gl.load().gl_rmsnorm(x, r, g, eps, rows, cols, sum, y, rstd, codes, scales, layout, None)


def _b(dy=16, s=16, g=16, rstd=16, dsum=None, rows=4, cols=128, dx=16, dg=16, ws=256, nbytes=1 << 30):
    return gl.load().gl_rmsnorm_bwd(dy, s, g, rstd, dsum, rows, cols, dx, dg, 0, ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(g=None), dict(y=None), dict(rows=-1), dict(cols=0), dict(eps=-1.0), dict(eps=float("nan")),
    dict(codes=16), dict(codes=16, scales=16, layout=2), dict(sum=32)])
def test_forward_invalid(kw):
    assert _c(**kw) == gl.GL_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(cols=12), dict(cols=16392), dict(x=8), dict(r=8), dict(g=8), dict(y=8),
    dict(sum=8), dict(rstd=2), dict(codes=4, scales=16), dict(cols=40, codes=16, scales=16),
    dict(cols=96, codes=16, scales=16, layout=1), dict(rows=1 << 31)])
def test_forward_unsupported(kw):
    assert _c(**kw) == gl.GL_ERR_UNSUPPORTED


def test_forward_without_rows_does_nothing():
    assert _c(x=None, y=None, rows=0) == gl.GL_OK


@pytest.mark.parametrize("kw", [dict(dy=None), dict(s=None), dict(g=None), dict(rstd=None), dict(dx=None),
                                dict(dg=None), dict(ws=None), dict(nbytes=4), dict(rows=-1), dict(cols=0)])
def test_backward_invalid(kw):
    assert _b(**kw) == gl.GL_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(dy=8), dict(s=8), dict(g=8), dict(dsum=8), dict(dx=8), dict(dg=8), dict(ws=128),
                                dict(rstd=2), dict(cols=20), dict(cols=16392)])
def test_backward_unsupported(kw):
    assert _b(**kw) == gl.GL_ERR_UNSUPPORTED


def test_workspace_size():
    lib = gl.load()
    assert lib.gl_rmsnorm_bwd_workspace_bytes(0, 128) == 128 * 4
    assert lib.gl_rmsnorm_bwd_workspace_bytes(5, 0) == 0
    assert lib.gl_rmsnorm_bwd_workspace_bytes(5, 12) == 0
    assert lib.gl_rmsnorm_bwd_workspace_bytes(1 << 20, 4096) % (4096 * 4) == 0


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("make", [
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5),                                    # not on a GPU
    lambda: gl.gl_rmsnorm(_z(4, 64, dtype=torch.float32), _z(64), 1e-5),               # dtype
    lambda: gl.gl_rmsnorm(_z(4, 128)[:, ::2], _z(64), 1e-5),                           # strided
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(32), 1e-5),                                    # gamma's shape
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5, residual=_z(3, 64)),                # residual's shape
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5, y=False),                           # no output
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5, mxfp8=True, mma_scales=True),       # 64 % 128
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5, out={"codes_r": _z(4, 64, dtype=U8)}),  # not asked for
    lambda: gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5, out={"y": _z(5, 64)}),
    lambda: gl.gl_rmsnorm(_z(64), _z(64), 1e-5),
    lambda: gl.gl_rmsnorm_bwd(_z(4, 64), _z(4, 64), _z(64), _z(4)),                    # rstd's dtype
    lambda: gl.gl_rmsnorm_bwd(_z(4, 64), _z(4, 64), _z(64), _z(4, dtype=torch.float32), accumulate=True),
    lambda: gl.gl_rmsnorm_bwd(_z(4, 64), _z(4, 60), _z(64), _z(4, dtype=torch.float32)),
])
def test_binding_refuses(make):
    with pytest.raises(gl.GlError):
        make()


def test_binding_names_what_it_refuses():
    rstd = _z(4, dtype=torch.float32)
    with pytest.raises(gl.GlError, match="workspace must be"):  # one byte, many times
        gl.gl_rmsnorm_bwd(_z(4, 64), _z(4, 64), _z(64), rstd, workspace=_z(1, dtype=U8).expand(1 << 20))
    with pytest.raises(gl.GlError, match="workspace must be"):
        gl.gl_rmsnorm_bwd(_z(4, 64), _z(4, 64), _z(64), rstd, workspace=1 << 20)
    with pytest.raises(gl.GlError, match="not a tensor"):
        gl.gl_rmsnorm(_z(4, 64), _z(64), 1e-5, out={"y": [0.0]})
