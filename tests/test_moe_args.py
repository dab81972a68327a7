"""What gl_moe_tokens refuses, before any CUDA call, and how its work is cut
(no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from grouped_gemm_splits_b200 import gl

W = gl.GlGrouped(gl.GL_STACKED, 16, None)
NOW = gl.GlGrouped(gl.GL_STACKED, None, None)


def _pg(n, p=16):
    arr = (ctypes.c_void_p * n)(*[p] * n)
    return gl.GlGrouped(gl.GL_PER_GROUP, None, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)))


def _m(x=16, router=16, w1=W, w2=W, act=gl.GL_ACT_SWIGLU, flags=1, T=4, E=8, k=2, H=64, F=32, idx=16, w=16, y=16,
       st=16, ws=256, nbytes=1 << 40, opts=None):
    return gl.load().gl_moe_tokens(x, router, w1, w2, act, flags, T, E, k, H, F, idx, w, y, st, ws, nbytes, opts, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w1=NOW), dict(w2=NOW), dict(idx=None), dict(w=None), dict(y=None), dict(st=None),
    dict(ws=None), dict(nbytes=100), dict(act=gl.GL_ACT_SILU), dict(act=7), dict(flags=2), dict(T=-1), dict(E=0),
    dict(k=0), dict(k=9), dict(H=0), dict(F=-8), dict(w1=_pg(8, None)),
    dict(opts=ctypes.pointer(gl.GlGemmOpts(gl.GL_TILES_SINGLE, 0, 0))),
    dict(opts=ctypes.pointer(gl.GlGemmOpts(gl.GL_TILES_PAIR, 0, 8)))])
def test_invalid(kw):
    assert _m(**kw) == gl.GL_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(T=129), dict(E=257), dict(E=32, k=17), dict(H=60), dict(F=20), dict(x=8), dict(router=8), dict(y=8),
    dict(ws=64), dict(idx=2), dict(w=2), dict(E=121, w1=_pg(121)), dict(E=121, w2=_pg(121)), dict(w1=_pg(8, 24))])
def test_unsupported(kw):
    assert _m(**kw) == gl.GL_ERR_UNSUPPORTED


def test_no_tokens_is_nothing_to_do():
    assert _m(T=0, x=None, idx=None, w=None, y=None) == gl.GL_OK


def test_workspace_size():
    f = gl.load().gl_moe_workspace_bytes
    assert f(129, 8, 2, 64, 32) == 0 and f(4, 8, 9, 64, 32) == 0 and f(4, 8, 2, 60, 32) == 0
    assert f(4, 8, 2, 64, 32) % 256 == 0
    # h (bf16) and the slots' second products (fp32) grow with the slots
    assert f(16, 8, 4, 640, 320) - f(16, 8, 2, 640, 320) == 2 * 16 * (640 * 4 + 320 * 2)


def test_every_block_has_one_owner():
    """The cut of a phase's blocks into CTA ranges, as the kernel computes it:
    contiguous, complete, and the owner formula names the range."""
    for total in (1, 2, 5, 147, 148, 149, 1000, 12345, 7 * 11 * 13):
        for ctas in (1, 2, 100, 148):
            n = min(total, ctas)
            begin = [total * c // n for c in range(n + 1)]
            assert begin[0] == 0 and begin[-1] == total and all(a < b for a, b in zip(begin, begin[1:]))
            owner = ((np.arange(total) + 1) * n - 1) // total
            for c in range(n):
                assert (owner[begin[c]:begin[c + 1]] == c).all()


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


ST = torch.zeros(1, dtype=torch.int32)


@pytest.mark.parametrize("make", [
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST, router_w=_z(4, 64)),  # not on a GPU
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST),                      # no routing
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST, router_w=_z(5, 64)),
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 16, 64), _z(4, 64, 16), 2, ST, router_w=_z(4, 64)),  # one factor only
    lambda: gl.gl_moe_tokens(_z(129, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST, router_w=_z(4, 64)),
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST.long(), router_w=_z(4, 64)),
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), [_z(64, 16)] * 3, 2, ST, router_w=_z(4, 64)),
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST, topk_idx=_z(2, 2, dtype=torch.int64),
                             topk_w=_z(2, 2, dtype=torch.float32)),
    lambda: gl.gl_moe_tokens(_z(2, 64), _z(4, 32, 64), _z(4, 64, 16), 2, ST, router_w=_z(4, 64), y=_z(3, 64)),
    lambda: gl.gl_moe_tokens(_z(2, 128)[:, ::2], _z(4, 32, 64), _z(4, 64, 16), 2, ST, router_w=_z(4, 64)),
])
def test_binding_refuses(make):
    with pytest.raises(gl.GlError):
        make()


@pytest.mark.parametrize("w1,w2,ws,why", [
    ([], [], None, "w1 must be"),
    (torch.tensor(0.0), _z(4, 64, 16), None, "w1 must be"),
    (_z(4, 32, 64), [], None, "w2 must be"),
    (_z(4, 32, 64), _z(16), None, "w2 must be"),
    (_z(4, 32, 64), _z(4, 64, 16), torch.zeros(1, dtype=torch.uint8).expand(1 << 24), "workspace must be"),
])
def test_binding_names_what_it_refuses(w1, w2, ws, why):
    with pytest.raises(gl.GlError, match=why):
        gl.gl_moe_tokens(_z(2, 64), w1, w2, 2, ST, router_w=_z(4, 64), workspace=ws)


@pytest.mark.parametrize("kw", [dict(H=(1 << 20) + 8), dict(F=(1 << 20) + 8), dict(st=18)])
def test_wide_layers_and_a_status_word_off_its_boundary_are_unsupported(kw):
    assert _m(**kw) == gl.GL_ERR_UNSUPPORTED


def test_the_widest_layer_has_a_workspace():
    f, n = gl.load().gl_moe_workspace_bytes, 1 << 20
    assert f(128, 256, 16, n, n) > 128 * 16 * (4 * n + 2 * n)
    assert f(1, 8, 2, n + 8, 64) == 0 and f(1, 8, 2, 64, n + 8) == 0
