"""What gl_fwd_act and gl_dgrad_act refuse, before any CUDA call (no GPU)."""
import ctypes

import pytest
import torch

from grouped_gemm_splits_b200 import gl

W = gl.GlGrouped(gl.GL_STACKED, 16, None)
NOW = gl.GlGrouped(gl.GL_STACKED, None, None)


def _f(x=16, w=W, bias=None, res=None, act=3, off=16, st=16, G=2, M=8, N=32, K=16, z=None, y=32, rows=8, opts=None):
    return gl.load().gl_fwd_act(x, w, bias, res, act, off, st, G, M, N, K, z, y, rows, opts, None)


def _d(dy=16, w=W, z=16, act=3, off=16, st=16, G=2, M=8, N=32, K=16, dz=32, rows=8, opts=None):
    return gl.load().gl_dgrad_act(dy, w, z, act, off, st, G, M, N, K, dz, rows, opts, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(w=NOW), dict(off=None), dict(st=None), dict(y=None), dict(rows=7),
                                dict(G=0), dict(G=4097), dict(N=0), dict(act=-1), dict(act=7), dict(z=32),
                                dict(z=48, res=48), dict(z=16), dict(y=16)])
def test_forward_invalid(kw):
    assert _f(**kw) == gl.GL_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(N=12), dict(K=12), dict(N=24, act=gl.GL_ACT_SWIGLU), dict(x=8), dict(y=40),
                                dict(z=8), dict(res=24)])
def test_forward_unsupported(kw):
    assert _f(**kw) == gl.GL_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dy=None), dict(w=NOW), dict(z=None), dict(off=None), dict(st=None), dict(dz=None),
                                dict(rows=7), dict(act=0), dict(act=7), dict(z=32), dict(dy=32), dict(G=0)])
def test_gradient_invalid(kw):
    assert _d(**kw) == gl.GL_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(N=12), dict(K=12), dict(dy=8), dict(z=8), dict(dz=40)])
def test_gradient_unsupported(kw):
    assert _d(**kw) == gl.GL_ERR_UNSUPPORTED


def test_no_rows_is_nothing_to_do():
    assert _f(M=0, x=None, y=None, rows=0) == gl.GL_OK
    assert _d(M=0, dy=None, z=None, dz=None, rows=0) == gl.GL_OK


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


OFF, ST = torch.zeros(3, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)


@pytest.mark.parametrize("make", [
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF, ST, gl.GL_ACT_SILU),               # not on a GPU
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF.int(), ST, gl.GL_ACT_SILU),
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF, ST.long(), gl.GL_ACT_SILU),
    lambda: gl.gl_fwd_act(_z(4, 16), _z(3, 32, 16), None, OFF, ST, gl.GL_ACT_SILU),
    lambda: gl.gl_fwd_act(_z(4, 16), [_z(32, 16)], None, OFF, ST, gl.GL_ACT_SILU),
    lambda: gl.gl_fwd_act(_z(4, 16), [_z(32, 16), _z(32, 8)], None, OFF, ST, gl.GL_ACT_SILU),
    lambda: gl.gl_fwd_act(_z(4, 16).float(), _z(2, 32, 16), None, OFF, ST, gl.GL_ACT_SILU),
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), _z(2, 16), OFF, ST, gl.GL_ACT_SWIGLU),        # bias has N columns
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF, ST, gl.GL_ACT_SWIGLU, residual=_z(4, 32)),
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF, ST, 9),
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF, ST, gl.GL_ACT_SILU, y=_z(3, 32)),
    lambda: gl.gl_fwd_act(_z(4, 16), _z(2, 32, 16), None, OFF, ST, gl.GL_ACT_SILU, z=_z(5, 32)),
    lambda: gl.gl_dgrad_act(_z(4, 32), _z(2, 32, 16), _z(4, 16), OFF, ST, gl.GL_ACT_NONE),
    lambda: gl.gl_dgrad_act(_z(4, 32), _z(2, 32, 16), _z(4, 16), OFF, ST, gl.GL_ACT_SWIGLU),      # z has 2K columns
    lambda: gl.gl_dgrad_act(_z(4, 16), _z(2, 32, 16), _z(4, 16), OFF, ST, gl.GL_ACT_SILU),        # dy has N columns
    lambda: gl.gl_dgrad_act(_z(4, 32), _z(2, 32, 16), _z(4, 16), OFF, ST, gl.GL_ACT_SILU, dz=_z(4, 32)),
])
def test_binding_refuses(make):
    with pytest.raises(gl.GlError):
        make()


@pytest.mark.parametrize("w", [[], _z(16), [None, None]])
def test_binding_names_the_weight_it_refuses(w):
    with pytest.raises(gl.GlError, match="w must be"):
        gl.gl_fwd_act(_z(4, 16), w, None, OFF, ST, gl.GL_ACT_SILU)
    with pytest.raises(gl.GlError, match="w must be"):
        gl.gl_dgrad_act(_z(4, 32), w, _z(4, 16), OFF, ST, gl.GL_ACT_SILU)


def _opts(tiles, wait=0, flags=0):
    return ctypes.pointer(gl.GlGemmOpts(tiles, wait, flags))


@pytest.mark.parametrize("tiles", [gl.GL_TILES_PAIR, gl.GL_TILES_SINGLE, gl.GL_TILES_BY_SIZE])
def test_tile_choices(tiles):
    """The library's choice can be combined with a wait bound (no rows: the arguments are checked, nothing launched)."""
    assert _f(M=0, rows=0, opts=_opts(tiles, 5000)) == gl.GL_OK
    assert _d(M=0, rows=0, opts=_opts(tiles, 5000)) == gl.GL_OK
    assert _f(M=0, rows=0, opts=_opts(3)) == gl.GL_ERR_INVALID
    assert _d(M=0, rows=0, opts=_opts(-1)) == gl.GL_ERR_INVALID


def test_calls_with_one_default_refuse_a_choice_by_size():
    lib, o = gl.load(), _opts(gl.GL_TILES_BY_SIZE)
    assert lib.gl_fwd(16, W, None, 16, 16, 2, 0, 32, 16, 16, 0, o, None) == gl.GL_ERR_INVALID
    assert lib.gl_dgrad(16, W, 16, 16, 2, 0, 32, 16, 16, 0, o, None) == gl.GL_ERR_INVALID
    assert lib.gl_wgrad(16, 16, 16, 16, 2, 0, 32, 16, W, 1, o, None) == gl.GL_ERR_INVALID
    assert lib.gl_moe_tokens(None, 16, W, W, gl.GL_ACT_SWIGLU, 0, 0, 8, 2, 64, 32, None, None, None, 16, 256, 1 << 40, o,
                             None) == gl.GL_ERR_INVALID


@pytest.mark.parametrize("pair,tiles", [(None, gl.GL_TILES_BY_SIZE), (True, gl.GL_TILES_PAIR),
                                        (False, gl.GL_TILES_SINGLE)])
def test_binding_keeps_the_choice_beside_a_wait_bound(pair, tiles):
    assert gl._opts_open(pair, 2000, 0).contents.tiles == tiles
    assert gl._opts_open(pair, 0, gl.GL_OPT_HOLD_LOADS).contents.tiles == tiles
