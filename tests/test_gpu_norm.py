"""gl_rmsnorm and gl_rmsnorm_bwd against the fp64 oracle (B200).

Tolerances: a bf16 result is off by half a step, 2^-8 of its value at most, a
code by half an E4M3 step.  The fp32 part adds the error of the row sum (its
terms are added in chains of at most 32 and then by trees of 10 levels: under
48 roundings of 2^-24, halved by the square root) and of a few products, so
2^-18 of the value covers it.
"""
import numpy as np
import pytest
import torch

from grouped_gemm_splits_b200 import gl
from oracle import block_oracle as blk
from oracle import gl_oracle as orc

from tests.gpu_util import SENTINEL_BF16, f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
F32 = 2.0 ** -18
EPS = 1e-5


def _rand(*shape, seed=0, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(BF).cuda()


def _close_bf16(got, ref):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= (2.0 ** -8 + F32) * np.abs(ref) + 1e-30), float(np.max(err / (np.abs(ref) + 1e-30)))


SHAPES = [(1, 8), (1, 16384), (3, 256), (5, 264), (33, 512), (130, 1024), (129, 1032), (257, 2048), (64, 4096),
          (19, 7168), (4, 12320), (2500, 640), (1300, 2176)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward_bf16(rows, cols, residual):
    x, gamma = _rand(rows, cols, seed=rows), _rand(cols, seed=cols, std=0.2, mean=1.0)
    r = _rand(rows, cols, seed=7, std=3.0) if residual else None
    out = gl.gl_rmsnorm(x, gamma, EPS, residual=r)
    s, rstd, y = blk.rmsnorm(f64(x), f64(r) if residual else None, f64(gamma), EPS)
    assert np.all(np.abs(f64(out["rstd"]) - rstd) <= F32 * rstd)
    _close_bf16(out["y"], y)
    if residual:
        _close_bf16(out["sum"], s)
    else:
        assert "sum" not in out


def _check_codes(codes, scales, y, mma):
    rows, cols = y.shape
    if mma:
        scales = scales.cpu().numpy()[orc.mma_offsets_rowwise(rows, cols)]
    else:
        scales = scales.cpu().numpy().reshape(rows, cols // 32)
    amax = np.abs(y).reshape(rows, cols // 32, 32).max(2)
    lo, hi = (orc.e8m0_exponent(amax * f) + 127 for f in (1 - F32, 1 + F32))
    assert np.all((scales >= lo) & (scales <= hi))
    step = 2.0 ** (scales.astype(np.float64) - 127)[:, :, None]
    got = orc.e4m3_decode(codes.cpu().numpy()).reshape(rows, cols // 32, 32)
    v = y.reshape(rows, cols // 32, 32) / step
    half = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-30))), -6) - 4)
    assert np.all(np.abs(got - v) <= half * (1 + 2.0 ** -10) + np.abs(v) * F32)


@pytest.mark.parametrize("rows,cols,mma", [(1, 32, False), (3, 96, False), (1, 128, True), (5, 384, True),
                                           (127, 1024, True), (129, 1152, True), (300, 2048, True),
                                           (33, 1056, False), (9, 7168, True), (2, 16384, True)])
@pytest.mark.parametrize("with_y", [False, True])
def test_forward_mxfp8(rows, cols, mma, with_y):
    x, r = _rand(rows, cols, seed=rows), _rand(rows, cols, seed=3, std=2.0)
    gamma = _rand(cols, seed=cols, std=0.5, mean=1.0)
    x[0, :32] = 0
    r[0, :32] = 0  # a block of zeros: scale byte 127, codes +-0 (the sign is gamma's)
    out = gl.gl_rmsnorm(x, gamma, EPS, residual=r, y=with_y, mxfp8=True, mma_scales=mma)
    s, _, y = blk.rmsnorm(f64(x), f64(r), f64(gamma), EPS)
    _check_codes(out["codes_r"], out["scales_r"], y, mma)
    assert ("y" in out) == with_y
    if with_y:
        _close_bf16(out["y"], y)
    _close_bf16(out["sum"], s)
    flat = out["scales_r"].cpu().numpy().reshape(-1)
    assert flat[0] == 127 and not (out["codes_r"][0, :32] & 0x7F).any()


# Without a residual a block takes rows two at a time, `grid` rows apart: row
# counts that end in the first or the second of them, and before the ring fills.
@pytest.mark.parametrize("rows,cols", [(1, 128), (2, 1024), (149, 4096), (297, 4096), (1037, 2048), (1776, 2048),
                                       (5000, 256), (4, 7168), (593, 7168), (741, 16384)])
def test_forward_without_residual(rows, cols):
    x, gamma = _rand(rows, cols, seed=rows), _rand(cols, seed=cols, std=0.5, mean=1.0)
    out = gl.gl_rmsnorm(x, gamma, EPS, mxfp8=True, mma_scales=True)
    _, rstd, y = blk.rmsnorm(f64(x), None, f64(gamma), EPS)
    assert np.all(np.abs(f64(out["rstd"]) - rstd) <= F32 * rstd)
    _close_bf16(out["y"], y)
    _check_codes(out["codes_r"], out["scales_r"], y, True)


@pytest.mark.parametrize("residual", [False, True])
def test_mean_squares_at_the_ends_of_fp32(residual):
    cols = 512
    x = torch.ones(6, cols, dtype=BF, device="cuda")
    x[0] = 2.0 ** 100  # the squares overflow: rstd is 0
    x[1] = 2.0 ** -100  # and vanish: eps decides
    x[2] = 2.0 ** 62  # their sum overflows: 512 * 2^124 = 2^133
    x[3] = 2.0 ** -62
    x[4] = 0.0
    gamma = torch.ones(cols, dtype=BF, device="cuda")
    r = torch.zeros_like(x) if residual else None
    for eps in (1e-5, 1e-38):
        out = gl.gl_rmsnorm(x, gamma, eps, residual=r)
        _, rstd, y = blk.rmsnorm(f64(x), None, f64(gamma), eps)
        over = (f64(x) ** 2).sum(1) >= 2.0 ** 128
        assert list(over) == [True, False, True, False, False, False]
        rstd[over], y[over] = 0, 0
        assert np.all(np.abs(f64(out["rstd"]) - rstd) <= F32 * rstd)
        _close_bf16(out["y"], y)


def test_bytes_of_absent_rows_and_outputs_not_asked_for_stay():
    rows, cols = 5, 256
    x, gamma = _rand(rows, cols), _rand(cols, mean=1.0)
    sc = torch.full((gl.mxfp8_scale_bytes(rows, cols, 1, False, True),), 0xAB, dtype=torch.uint8, device="cuda")
    gl.gl_rmsnorm(x, gamma, EPS, y=False, mxfp8=True, mma_scales=True, out={"scales_r": sc})
    at = orc.mma_offsets_rowwise(rows, cols).reshape(-1)
    rest = np.setdiff1d(np.arange(sc.numel()), at)
    assert np.all(sc.cpu().numpy()[rest] == 0xAB)


def test_rows_of_a_larger_buffer_stay():
    big = torch.full((8, 512), SENTINEL_BF16, dtype=torch.int16, device="cuda").view(BF)
    x, gamma = _rand(5, 512), _rand(512, mean=1.0)
    gl.gl_rmsnorm(x, gamma, EPS, out={"y": big[:5]})
    assert (big[5:].view(torch.int16) == SENTINEL_BF16).all()


@pytest.mark.parametrize("cols", [512, 4096])
def test_in_place(cols):
    x, r, gamma = _rand(70, cols), _rand(70, cols, seed=1), _rand(cols, seed=2, mean=1.0)
    want = gl.gl_rmsnorm(x, gamma, EPS, residual=r)
    x2, r2 = x.clone(), r.clone()
    got = gl.gl_rmsnorm(x2, gamma, EPS, residual=r2, out={"sum": r2, "y": x2})
    assert torch.equal(x2, want["y"]) and torch.equal(r2, want["sum"]) and torch.equal(got["rstd"], want["rstd"])


def test_zero_rows_nan_and_infinity():
    x, gamma = _rand(6, 256), _rand(256, mean=1.0)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    out = gl.gl_rmsnorm(x, gamma, EPS, mxfp8=True)
    y = f64(out["y"])
    assert not y[1].any() and np.isnan(y[2]).all()
    assert np.isnan(y[3, 7]) and not np.delete(y[3], 7).any()
    assert np.isfinite(y[[0, 4, 5]]).all()
    assert np.isnan(orc.e4m3_decode(out["codes_r"].cpu().numpy())[2]).all()
    e = gl.gl_rmsnorm(x[:0], gamma, EPS, mxfp8=True, mma_scales=True)
    assert e["y"].shape == (0, 256)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dsum,accumulate", [(False, False), (True, True)])
def test_backward(rows, cols, dsum, accumulate):
    s, dy, gamma = _rand(rows, cols, seed=1, std=2.0), _rand(rows, cols, seed=2), _rand(cols, seed=3, mean=1.0)
    ds = _rand(rows, cols, seed=4) if dsum else None
    rstd = torch.rsqrt(s.float().square().mean(1) + EPS)
    old = torch.randn(cols, generator=torch.Generator().manual_seed(8)).cuda() if accumulate else None
    dx, dg = gl.gl_rmsnorm_bwd(dy, s, gamma, rstd, dsum=ds, dgamma=old.clone() if accumulate else None,
                               accumulate=accumulate)
    rdx, rdg = blk.rmsnorm_bwd(f64(dy), f64(s), f64(gamma), f64(rstd), f64(ds) if dsum else None)
    # dx is a difference: its fp32 error is relative to the terms, not to the result
    xh = np.abs(f64(s) * f64(rstd)[:, None])
    g = np.abs(f64(dy) * f64(gamma))
    terms = f64(rstd)[:, None] * (g + xh * np.mean(g * xh, axis=1, keepdims=True)) + (np.abs(f64(ds)) if dsum else 0)
    assert np.all(np.abs(f64(dx) - rdx) <= 2.0 ** -8 * np.abs(rdx) + F32 * terms)
    scale = np.sum(np.abs(f64(dy)) * xh, axis=0) + (np.abs(f64(old)) if accumulate else 0)
    # the longest chain of fp32 additions: a block's rows, then the blocks'
    steps = 16 + rows
    assert np.all(np.abs(f64(dg) - rdg - (f64(old) if accumulate else 0)) <= steps * 2.0 ** -24 * scale + 1e-30)


def test_backward_without_rows():
    gamma, dg = _rand(256), torch.ones(256, device="cuda")
    e, z = _rand(0, 256), torch.zeros(0, device="cuda")
    gl.gl_rmsnorm_bwd(e, e, gamma, z, dgamma=dg, accumulate=True)
    assert (dg == 1).all()
    gl.gl_rmsnorm_bwd(e, e, gamma, z, dgamma=dg)
    assert (dg == 0).all()


def test_backward_is_deterministic_and_in_place_over_a_dirty_workspace():
    s, dy, gamma = _rand(3000, 1536, seed=1), _rand(3000, 1536, seed=2), _rand(1536, mean=1.0)
    rstd = torch.rsqrt(s.float().square().mean(1) + EPS)
    ws = torch.full((gl.rmsnorm_bwd_workspace_bytes(3000, 1536),), 0xFF, dtype=torch.uint8, device="cuda")
    a = gl.gl_rmsnorm_bwd(dy, s, gamma, rstd, dsum=dy)
    d2 = dy.clone()
    b = gl.gl_rmsnorm_bwd(d2, s, gamma, rstd, dsum=dy, dx=d2, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_forward_output_feeds_the_mxfp8_product_and_graph_replay():
    """norm -> MXFP8 -> grouped product, captured on a side stream and replayed on new inputs."""
    M, K, N, G = 300, 256, 384, 3
    m = torch.tensor([100, 0, 200], device="cuda")
    off, st = gl.gl_offsets(m, M)
    w = _rand(G, N, K, seed=9, std=0.06)
    gamma = _rand(K, seed=3, std=0.1, mean=1.0)
    qw = gl.group_quantize_mxfp8(w, rowwise=True, mma_scales=True)
    x = _rand(M, K, seed=1)

    def step():
        q = gl.gl_rmsnorm(x, gamma, EPS, y=False, mxfp8=True, mma_scales=True)
        return gl.gl_fwd_mxfp8(q["codes_r"], q["scales_r"], qw["codes_r"].view(G, N, K), qw["scales_r"], None, off, st)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    x.copy_(_rand(M, K, seed=2))
    graph.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _, _, n = blk.rmsnorm(f64(x), None, f64(gamma), EPS)
    wq, ws = orc.quantize_rowwise(f64(w).reshape(G * N, K))
    wd = orc.dequant_rowwise(wq, ws).reshape(G, N, K)
    nq, ns = orc.quantize_rowwise(n)
    ref = np.zeros((M, N))
    nd = orc.dequant_rowwise(nq, ns)
    ref[:100], ref[100:] = nd[:100] @ wd[0].T, nd[100:] @ wd[2].T
    assert orc.rel_frobenius(f64(y), ref) <= 1e-2


def test_backward_captured_and_replayed():
    """Two captured backward passes in one graph, each with its own workspace, follow new inputs."""
    rows, cols = 700, 1040
    s, dy, gamma = _rand(rows, cols, seed=1), _rand(rows, cols, seed=2), _rand(cols, seed=3, mean=1.0)
    rstd = torch.rsqrt(s.float().square().mean(1) + EPS)
    dg = torch.zeros(cols, device="cuda")

    def step(dg):
        dx, _ = gl.gl_rmsnorm_bwd(dy, s, gamma, rstd, dgamma=dg, accumulate=True)
        return gl.gl_rmsnorm_bwd(dx, s, gamma, rstd, dsum=dy, dgamma=dg, accumulate=True)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(torch.zeros_like(dg))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(dg)
    total = torch.zeros_like(dg)
    for seed in (7, 8):
        dy.copy_(_rand(rows, cols, seed=seed))
        graph.replay()
        assert torch.equal(out, step(total)) and torch.equal(dg, total)


def test_more_than_two_to_the_31_elements():
    """Offsets past 32 bits: the last rows of 300000 x 8192 (4.9 GB a tensor)."""
    rows, cols, last = 300000, 8192, 5
    x, gamma = torch.zeros(rows, cols, dtype=BF, device="cuda"), _rand(cols, seed=3, mean=1.0)
    x[-last:] = _rand(last, cols, seed=1)
    out = gl.gl_rmsnorm(x, gamma, EPS, mxfp8=True)
    s, rstd, y = blk.rmsnorm(f64(x[-last:]), None, f64(gamma), EPS)
    _close_bf16(out["y"][-last:], y)
    _check_codes(out["codes_r"][-last:], out["scales_r"][-last:], y, False)
    assert not out["y"][:last].any()
    del out["codes_r"]
    dx, dg = gl.gl_rmsnorm_bwd(x, x, gamma, out["rstd"], dx=out["y"])
    rdx, _ = blk.rmsnorm_bwd(s, s, f64(gamma), f64(out["rstd"][-last:]), None)
    assert orc.rel_frobenius(f64(dx[-last:]), rdx) <= 5e-3
    assert not dx[:last].any()
