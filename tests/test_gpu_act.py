"""gl_fwd_act and gl_dgrad_act against the fp64 oracle (B200).

Elementwise tolerance: half a bf16 step (2^-8 of the value) for the final
rounding, plus what the product's fp32 sum may be off by, carried through the
activation.  A sum of K products in K / 16 tensor-core steps, each off by at
most one fp32 unit of the largest partial sum, is within (K / 16 + 16) * 2^-23
of sum |x w|.  The activations' own fp32 error (fast exponential and division:
a few units, on values below |u|) is taken as 2^-18 (1 + |u|).  No slope
here exceeds 1.13, but relu2's, 2 |u|.
"""
import numpy as np
import pytest
import torch

from grouped_gemm_splits_b200 import gl, synth
from oracle import block_oracle as blk
from oracle import gl_oracle as orc
from tests.gpu_util import f64, offsets_on_device, sentinel_like, untouched

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8


def _rand(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def _sum_error(K, x, w, m):
    return (K / 16 + 16) * 2.0 ** -23 * orc.fwd(np.abs(x), np.abs(w), None, m)


def _value_error(name, u, du):
    """How far an activation's value is off when u is off by du, with its own fp32 error."""
    lip = 2 * np.abs(u) + du if name == "relu2" else 1.13
    own = 2.0 ** -18 * (np.abs(u) + (u * u if name == "relu2" else 1))
    return lip * du + own


def _check(got, ref, tol):
    err = np.abs(f64(got) - ref)
    bound = HALF * np.abs(ref) + tol * (1 + HALF) + 1e-30
    assert np.all(err <= bound), float(np.max(err / bound))


CASES = [  # splits, K, N
    ([1], 8, 16), ([0, 3, 0, 130, 1], 136, 48), ([257, 0, 255], 512, 272), ([0, 96, 160, 256], 128, 256),
    ([77, 300, 5], 1000, 528), ([640], 64, 1040),
]


@pytest.mark.parametrize("m,K,N", CASES)
@pytest.mark.parametrize("name", blk.ACTS)
@pytest.mark.parametrize("bias,residual,pair", [(False, False, None), (True, True, True), (True, True, False)])
def test_forward(m, K, N, name, bias, residual, pair):
    G, M = len(m), sum(m)
    x, w = _rand(M, K, seed=1), _rand(G, N, K, seed=2, std=2.0 / np.sqrt(K))
    b = _rand(G, N, seed=3) if bias else None
    nout = N // 2 if name in blk.GATED else N
    r = _rand(M, nout, seed=4, std=2.0) if residual else None
    off, st = offsets_on_device(m, M)
    y = sentinel_like(M + 3, nout)
    y, z = gl.gl_fwd_act(x, w, b, off, st, gl.ACTS[name], residual=r, save_z=True, y=y, pair=pair)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and untouched(y[M:])
    ref, u = blk.fwd_act(f64(x), f64(w), f64(b) if bias else None, m, name, f64(r) if residual else None)
    du = _sum_error(K, f64(x), f64(w), m) + 2.0 ** -23 * np.abs(u)
    _check(z, u, du)
    if name in blk.GATED:
        F = nout
        inner = blk.GATED[name]
        a, da = blk.act(inner, u[:, :F]), _value_error(inner, u[:, :F], du[:, :F])
        tol = np.abs(a) * du[:, F:] + da * (np.abs(u[:, F:]) + du[:, F:])
    else:
        tol = _value_error(name, u, du)
    _check(y[:M], ref, tol + 2.0 ** -23 * np.abs(ref))
    # without z the outputs are the same bits
    again, none = gl.gl_fwd_act(x, w, b, off, st, gl.ACTS[name], residual=r, pair=pair)
    assert none is None and torch.equal(again, y[:M])


@pytest.mark.parametrize("m,K,N", CASES)
@pytest.mark.parametrize("name", blk.ACTS[1:])
@pytest.mark.parametrize("pair", [True, False])
def test_gradient(m, K, N, name, pair):
    K, N = N, K  # the contraction runs over N here
    G, M = len(m), sum(m)
    two = 2 if name in blk.GATED else 1
    dy, w = _rand(M, N, seed=1), _rand(G, N, K, seed=2, std=2.0 / np.sqrt(N))
    z = _rand(M, K * two, seed=3, std=2.0)
    off, st = offsets_on_device(m, M)
    dz = gl.gl_dgrad_act(dy, w, z, off, st, gl.ACTS[name], dz=sentinel_like(M + 2, K * two), pair=pair)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and untouched(dz[M:])
    ref = blk.dgrad_act(f64(dy), f64(w), m, name, f64(z))
    dh = orc.dgrad(f64(dy), f64(w), m)
    ddh = (N / 16 + 16) * 2.0 ** -23 * orc.dgrad(np.abs(f64(dy)), np.abs(f64(w)), m)
    zz = f64(z)
    inner = blk.GATED.get(name, name)
    z0 = zz[:, :K]
    sl = np.abs(blk.slope(inner, z0))
    # q(1 - q) keeps an absolute error of a few 2^-24, multiplied by |u| <= 16 or so
    dsl = 2.0 ** -17 * (1 + np.abs(z0))
    if two == 2:
        z1 = np.abs(zz[:, K:])
        a = np.abs(blk.act(inner, z0))
        tol = np.concatenate([z1 * (ddh * (sl + dsl) + np.abs(dh) * dsl),
                              ddh * a + (np.abs(dh) + ddh) * 2.0 ** -18 * (1 + np.abs(z0))], axis=1)
    else:
        tol = ddh * (sl + dsl) + np.abs(dh) * dsl
    _check(dz[:M], ref, tol)


@pytest.mark.parametrize("width", [8, 24, 136])
@pytest.mark.parametrize("pair", [True, False])
def test_rows_that_are_no_multiple_of_32_bytes(width, pair):
    """Widths that are odd multiples of 8, and buffers that start 16 bytes past a 32-byte boundary."""
    m, K = [70, 0, 3, 190], 40
    M, G = sum(m), len(m)
    x, w, b = _rand(M, K, seed=1), _rand(G, width, K, seed=2, std=0.3), _rand(G, width, seed=3)
    r = _rand(M, width, seed=4)
    off, st = offsets_on_device(m, M)
    y, z = gl.gl_fwd_act(x, w, b, off, st, gl.GL_ACT_GELU, residual=r, save_z=True, pair=pair)
    ref, u = blk.fwd_act(f64(x), f64(w), f64(b), m, "gelu", f64(r))
    du = _sum_error(K, f64(x), f64(w), m) + 2.0 ** -23 * np.abs(u)
    _check(z, u, du)
    _check(y, ref, _value_error("gelu", u, du) + 2.0 ** -23 * np.abs(ref))
    dy = _rand(M, K, seed=5)
    w2 = _rand(G, K, width, seed=6, std=0.3)
    for name, two in (("silu", 1), ("swiglu", 2), ("geglu", 2)):
        zz = _rand(M, width * two, seed=7)
        dz = gl.gl_dgrad_act(dy, w2, zz, off, st, gl.ACTS[name], pair=pair)
        ref = blk.dgrad_act(f64(dy), f64(w2), m, name, f64(zz))
        # |value|, |slope| and the other factor are below 6 here
        ddh = (K / 16 + 16) * 2.0 ** -23 * orc.dgrad(np.abs(f64(dy)), np.abs(f64(w2)), m)
        tol = 36 * (ddh + 2.0 ** -16 * (1 + np.abs(orc.dgrad(f64(dy), f64(w2), m))))
        _check(dz, ref, np.concatenate([tol] * two, axis=1))
    # the same bits through buffers off the 32-byte boundary
    w16 = _rand(G, 32, K, seed=8, std=0.3)
    want, wz = gl.gl_fwd_act(x, w16, None, off, st, gl.GL_ACT_SWIGLU, residual=_rand(M, 16, seed=9), save_z=True, pair=pair)

    def shifted(rows, cols):
        t = torch.zeros(rows * cols + 8, dtype=BF, device="cuda")[8:].view(rows, cols)
        assert t.data_ptr() % 32 == 16
        return t

    res = shifted(M, 16)
    res.copy_(_rand(M, 16, seed=9))
    got, gz = gl.gl_fwd_act(x, w16, None, off, st, gl.GL_ACT_SWIGLU, residual=res, z=shifted(M, 32), y=shifted(M, 16),
                            pair=pair)
    assert torch.equal(got, want) and torch.equal(gz, wz)
    assert int(st.item()) == 0


@pytest.mark.parametrize("name", ["none", "relu", "relu2"])
def test_integers_are_exact(name):
    m, K, N = [100, 0, 300, 7], 96, 264
    d = {k: v.cuda() for k, v in synth.integer_operands(4, 407, N, K, 5).items()}
    off, st = offsets_on_device(m, 407)
    w = d["w"] * (torch.arange(K, device="cuda") < 8)  # |u| <= 16: its square stays exact in bf16
    w = w.to(BF).contiguous()
    r = torch.randint(-64, 65, (407, N), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    y, z = gl.gl_fwd_act(d["x"], w, d["bias"], off, st, gl.ACTS[name], residual=r, save_z=True)
    ref, u = blk.fwd_act(f64(d["x"]), f64(w), f64(d["bias"]), m, name, f64(r))
    assert np.array_equal(f64(z), u)
    exact = np.abs(ref) <= 256
    assert np.array_equal(f64(y)[exact], ref[exact])


def test_per_group_weights_and_more_groups_than_one_launch():
    G, K, N = 70, 64, 96
    m = [(i * 7) % 5 * 9 for i in range(G)]
    M = sum(m)
    x, w, b = _rand(M, K), _rand(G, N, K, seed=1, std=0.2), _rand(G, N, seed=2)
    off, st = offsets_on_device(m, M)
    for act in (gl.GL_ACT_GELU, gl.GL_ACT_SWIGLU):
        want, wz = gl.gl_fwd_act(x, w, b, off, st, act, save_z=True)
        got, z = gl.gl_fwd_act(x, [w[g].clone() for g in range(G)], [b[g].clone() for g in range(G)], off, st, act,
                               save_z=True)
        assert torch.equal(want, got) and torch.equal(wz, z)
    zz, dy = _rand(M, 2 * K, seed=3), _rand(M, N, seed=4)
    assert torch.equal(gl.gl_dgrad_act(dy, w, zz, off, st, gl.GL_ACT_GEGLU),
                       gl.gl_dgrad_act(dy, [w[g].clone() for g in range(G)], zz, off, st, gl.GL_ACT_GEGLU))


def test_none_is_the_plain_product():
    m, K, N = [90, 0, 41], 200, 520
    x, w, b = _rand(131, K), _rand(3, N, K, seed=1, std=0.1), _rand(3, N, seed=2)
    off, st = offsets_on_device(m, 131)
    assert torch.equal(gl.gl_fwd_act(x, w, b, off, st, gl.GL_ACT_NONE)[0], gl.gl_fwd(x, w, b, off, st))


def test_residual_in_place_and_status():
    m, K, N = [200, 100], 128, 256
    x, w, r = _rand(300, K), _rand(2, N, K, seed=1, std=0.1), _rand(300, N, seed=2)
    off, st = offsets_on_device(m, 300)
    want, _ = gl.gl_fwd_act(x, w, None, off, st, gl.GL_ACT_SILU, residual=r)
    buf = r.clone()
    gl.gl_fwd_act(x, w, None, off, st, gl.GL_ACT_SILU, residual=buf, y=buf)
    assert torch.equal(buf, want)
    off, st = offsets_on_device([200, 99], 300)  # the sizes do not add up: nothing is written
    y, z, dz = sentinel_like(300, N), sentinel_like(300, N), sentinel_like(300, K)
    gl.gl_fwd_act(x, w, None, off, st, gl.GL_ACT_SILU, z=z, y=y)
    gl.gl_dgrad_act(r, w, x, off, st, gl.GL_ACT_SILU, dz=dz)
    assert untouched(y) and untouched(z) and untouched(dz) and int(st.item()) == gl.GL_DEV_SUM_MISMATCH


def test_a_wait_that_runs_out_is_reported():
    x, w = _rand(64, 64), _rand(1, 64, 64, seed=1)
    off, st = offsets_on_device([64], 64)
    y = sentinel_like(64, 32)
    gl.gl_fwd_act(x, w, None, off, st, gl.GL_ACT_SWIGLU, y=y, wait_limit_us=2000, opt_flags=gl.GL_OPT_HOLD_LOADS)
    torch.cuda.synchronize()
    assert int(st.item()) == gl.GL_DEV_TIMEOUT and untouched(y)


def test_large_and_special_values():
    """Far arguments saturate, a NaN stays a NaN in its own element."""
    K = N = 64
    x = torch.zeros(128, K, dtype=BF, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(1, N, K, dtype=BF, device="cuda")
    vals = [0.0, -0.0, 1e4, -1e4, 1e30, -1e30, 88.0, -88.0, 100.0, -100.0]
    w[0, :len(vals), 0] = torch.tensor(vals, dtype=BF, device="cuda")
    off, st = offsets_on_device([128], 128)
    for name in ("gelu", "silu", "relu"):
        y, z = gl.gl_fwd_act(x, w, None, off, st, gl.ACTS[name], save_z=True)
        ref = blk.act("relu", f64(z)[0, :len(vals)])
        got = f64(y)[0, :len(vals)]
        assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + 1e-30)
        zz = z.clone()
        zz[0, 20] = float("nan")
        eye = torch.eye(64, device="cuda").to(BF).view(1, 64, 64)
        dz = f64(gl.gl_dgrad_act(torch.ones(128, 64, dtype=BF, device="cuda"), eye, zz, off, st, gl.ACTS[name]))
        far = [2, 3, 4, 5, 6, 7, 8, 9]
        assert np.array_equal(dz[0, far], (f64(z)[0, far] > 0).astype(float))
        if name != "relu":
            assert np.isnan(dz[0, 20])
        assert np.isfinite(np.delete(dz[0], 20)).all() and np.isfinite(dz[1:]).all()


def test_expert_block_forward_and_backward():
    """norm -> gated product -> second product with the residual, and all of its gradients, against fp64 autograd."""
    m = [130, 0, 257, 61]
    M, H, F, G = 448, 256, 192, 4
    x, gamma = _rand(M, H, seed=1), (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(2))).to(BF).cuda()
    w1, w2 = _rand(G, 2 * F, H, seed=3, std=H ** -0.5), _rand(G, H, F, seed=4, std=F ** -0.5)
    b1, dout = _rand(G, 2 * F, seed=5, std=0.1), _rand(M, H, seed=6)
    off, st = offsets_on_device(m, M)
    act = gl.GL_ACT_SWIGLU

    n = gl.gl_rmsnorm(x, gamma, 1e-5)
    h, z = gl.gl_fwd_act(n["y"], w1, b1, off, st, act, save_z=True)
    out, _ = gl.gl_fwd_act(h, w2, None, off, st, gl.GL_ACT_NONE, residual=x)
    dz = gl.gl_dgrad_act(dout, w2, z, off, st, act)
    dw2 = gl.gl_wgrad(h, dout, off, st, torch.zeros(G, H, F, device="cuda"))
    dn = gl.gl_dgrad(dz, w1, off, st)
    dw1 = gl.gl_wgrad(n["y"], dz, off, st, torch.zeros(G, 2 * F, H, device="cuda"))
    db1 = gl.gl_dbias(dz, off, st)
    dx, dgamma = gl.gl_rmsnorm_bwd(dn, x, gamma, n["rstd"], dsum=dout)
    assert int(st.item()) == 0

    leaves = {k: v.double().cpu().requires_grad_() for k, v in
              dict(x=x, gamma=gamma, w1=w1, w2=w2, b1=b1).items()}
    X = leaves["x"]
    N = X / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-5) * leaves["gamma"]
    o = [0, 130, 130, 387, 448]
    rows = []
    for g in range(G):
        u = N[o[g]:o[g + 1]] @ leaves["w1"][g].T + leaves["b1"][g]
        rows.append((torch.nn.functional.silu(u[:, :F]) * u[:, F:]) @ leaves["w2"][g].T)
    Y = torch.cat(rows) + X
    (Y * dout.double().cpu()).sum().backward()
    got = dict(x=dx, gamma=dgamma, w1=dw1, w2=dw2, b1=db1)
    # four bf16 roundings (2^-8 each at most, 2^-9.8 on average) lie between the leaves and the results
    assert orc.rel_frobenius(f64(out), Y.detach().numpy()) <= 5e-3
    for k, v in got.items():
        assert orc.rel_frobenius(f64(v), leaves[k].grad.numpy()) <= 1e-2, k


def test_captured_and_replayed_on_another_stream():
    m = torch.tensor([50, 30, 20], device="cuda")
    x, w, r = _rand(100, 64), _rand(3, 96, 64, seed=1, std=0.2), _rand(100, 48, seed=2)

    def step():
        off, st = gl.gl_offsets(m, 100)
        y, z = gl.gl_fwd_act(x, w, None, off, st, gl.GL_ACT_GEGLU, residual=r, save_z=True)
        return y, z

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = step()
    for sizes in ([0, 100, 0], [33, 33, 34]):
        m.copy_(torch.tensor(sizes))
        x.copy_(_rand(100, 64, seed=sizes[0]))
        graph.replay()
        want_y, want_z = step()
        assert torch.equal(y, want_y) and torch.equal(z, want_z)


def test_more_than_two_to_the_31_elements():
    """Offsets past 32 bits: the last rows of y and z, 300000 x 8192 and 300000 x 16384."""
    M, K, F, last = 300000, 16, 8192, 4
    x, w = torch.zeros(M, K, dtype=BF, device="cuda"), _rand(2, 2 * F, K, seed=1)
    x[-last:] = _rand(last, K, seed=2)
    off, st = offsets_on_device([M - 3, 3], M)
    y, z = gl.gl_fwd_act(x, w, None, off, st, gl.GL_ACT_SWIGLU, save_z=True)
    m = [last - 3, 3]
    ref, u = blk.fwd_act(f64(x[-last:]), f64(w), None, m, "swiglu", None)
    assert orc.rel_frobenius(f64(y[-last:]), ref) <= 5e-3 and orc.rel_frobenius(f64(z[-last:]), u) <= 5e-3
    assert not y[:last].any() and not z[:last].any()
    del y
    z[:-last] = 0
    dy = torch.zeros(M, K, dtype=BF, device="cuda")
    dy[-last:] = _rand(last, K, seed=3)
    w2 = _rand(2, K, F, seed=4)
    dz = gl.gl_dgrad_act(dy, w2, z, off, st, gl.GL_ACT_SWIGLU)
    assert orc.rel_frobenius(f64(dz[-last:]), blk.dgrad_act(f64(dy[-last:]), f64(w2), m, "swiglu", f64(z[-last:]))) <= 5e-3
    assert not dz[:last].any() and int(st.item()) == 0


def _sigmoid(v):
    return np.where(v < 0, np.exp(-np.abs(v)), 1.0) / (1 + np.exp(-np.abs(v)))


@pytest.mark.parametrize("name", ["silu", "gelu", "swiglu"])
def test_far_negative_arguments(name):
    """Values down to bf16's smallest: e^-88 is past 2^126, and e^-89 past fp32's largest value, but u e^u is not 0.

    Half a bf16 step (2^-8 relative; 2^-134 below bf16's normal range); the exponential's argument, 97 at most, is off by
    three fp32 roundings (3 * 97 * 2^-24 < 2^-15, relative in the value); its subnormal results by 2^-150, times |u|;
    and the last two bits of the fast forms, 2^-20.
    """
    u = np.concatenate([np.arange(-97.0, -79.9, 0.5), [-20.0, -5.0, -0.5, 0.0, 3.0]])
    if name == "gelu":
        u = np.concatenate([np.arange(-10.5, -9.0, 0.0625), [-3.0, -0.5, 0.0, 3.0]])
    n, K = len(u), 64
    width = 64
    x = torch.zeros(3, K, dtype=BF, device="cuda")
    x[:, 0] = 1
    gated = name == "swiglu"
    w = torch.zeros(1, width * (2 if gated else 1), K, dtype=BF, device="cuda")
    w[0, :n, 0] = torch.tensor(u, dtype=BF, device="cuda")
    if gated:
        w[0, width:, 0] = 1
    u = f64(w)[0, :n, 0]
    off, st = offsets_on_device([3], 3)
    y, z = gl.gl_fwd_act(x, w, None, off, st, gl.ACTS[name], save_z=True)
    assert np.array_equal(f64(z)[0, :n], u)
    c = 2 * np.sqrt(2 / np.pi)
    v, dv = (c * (u + 0.044715 * u ** 3), c * (1 + 3 * 0.044715 * u * u)) if name == "gelu" else (u, 1.0)
    q = _sigmoid(v)
    rel, least = 2.0 ** -8 + 2.0 ** -15 + 2.0 ** -20, 2.0 ** -134 + np.abs(u) * 2.0 ** -150
    ref = u * q
    assert np.all(np.abs(f64(y)[:, :n] - ref) <= rel * np.abs(ref) + least)
    assert np.all(f64(y)[0, :n][(u < 0) & (ref < -2.0 ** -130)] < 0)
    # slope q + u q (1 - q) v'(u): its two terms are off like the value; silu's is 0 where q is below 2^-126
    eye = torch.eye(width, device="cuda").to(BF).view(1, width, width)
    dz = f64(gl.gl_dgrad_act(torch.ones(3, width, dtype=BF, device="cuda"), eye, z, off, st, gl.ACTS[name]))
    if gated:  # the other factor's gradient: the value
        assert np.all(np.abs(dz[:, width:width + n] - ref) <= rel * np.abs(ref) + least)
    dz = dz[:, :n]
    qs = q if name == "gelu" else np.where(q < 2.0 ** -126, 0, q)
    first, second = qs, u * qs * _sigmoid(-v) * dv
    bound = 2.0 ** -8 * np.abs(first + second) + (rel - 2.0 ** -8) * (np.abs(first) + np.abs(second)) \
        + 2.0 ** -134 + (1 + np.abs(u * dv)) * 2.0 ** -149
    assert np.all(np.abs(dz - (first + second)) <= bound)
    assert int(st.item()) == 0


@pytest.mark.parametrize("name", blk.ACTS[1:])
def test_a_nan_goes_through_every_gradient(name):
    """A NaN pre-activation makes its own gradient NaN, whatever the activation, and no other one."""
    M, K, N = 40, 64, 32
    two = 2 if name in blk.GATED else 1
    dy, w, z = _rand(M, N, seed=1), _rand(1, N, K, seed=2, std=0.3), _rand(M, two * K, seed=3)
    z[5, 20] = z[39, 0] = float("nan")
    off, st = offsets_on_device([M], M)
    nan = np.zeros((M, two * K), dtype=bool)
    nan[5, 20] = nan[39, 0] = True
    if two == 2:  # the value is the other factor's slope
        nan[5, K + 20] = nan[39, K] = True
    for pair in (True, False):
        assert np.array_equal(np.isnan(f64(gl.gl_dgrad_act(dy, w, z, off, st, gl.ACTS[name], pair=pair))), nan)
    assert int(st.item()) == 0


@pytest.mark.parametrize("M,K,N,act", [(1025, 7168, 4096, gl.GL_ACT_SWIGLU), (1025, 14336, 4096, gl.GL_ACT_NONE)])
def test_the_tile_shape_chosen_for_one_group(M, K, N, act):
    """One group's tiles are known exactly: five rows of 256-row tiles do not fit a wave of pairs here, nine of 128-row
    tiles fit one of single CTAs, and pairs take half as long again.  (Times in turn, medians; the choice may be off by
    a quarter.)"""
    x, w = _rand(M, K), _rand(1, N, K, seed=1, std=0.02)
    off, st = offsets_on_device([M], M)
    graphs = {}
    for pair in (None, True, False):
        gl.gl_fwd_act(x, w, None, off, st, act, pair=pair)
        torch.cuda.synchronize()
        graphs[pair] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[pair]):
            for _ in range(10):
                gl.gl_fwd_act(x, w, None, off, st, act, pair=pair)
    times = {pair: [] for pair in graphs}
    for _ in range(9):
        for pair, graph in graphs.items():
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            times[pair].append(begin.elapsed_time(end))
    took = {pair: sorted(t)[4] for pair, t in times.items()}
    assert took[None] <= 1.25 * min(took[True], took[False]), took
    assert int(st.item()) == 0
