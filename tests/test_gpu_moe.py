"""gl_moe_tokens against the fp64 oracle (B200).

Logits: products of bf16 summed in fp32, within (H / 16 + 16) * 2^-23 of
sum |x r|; two experts closer than twice that may trade places, others not.
Weights: e^l has the logits' error as its relative error, twice (numerator and
sum).  y: half a bf16 step of its value, plus half a step of every h carried
through the second product (worst case, elementwise), and the library's
relative Frobenius bound of 5e-3 per token (typical roundings).
"""
import numpy as np
import pytest
import torch

from grouped_gemm_splits_b200 import gl
from oracle import block_oracle as blk
from oracle import gl_oracle as orc
from tests.gpu_util import TOL_BF16, f64, sentinel_like, untouched

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _layer(T, E, H, F, seed=0):
    return (_rand(T, H, seed=seed), _rand(E, H, seed=seed + 1, std=H ** -0.5),
            _rand(E, 2 * F, H, seed=seed + 2, std=H ** -0.5), _rand(E, H, F, seed=seed + 3, std=F ** -0.5))


def _check_y(y, x, idx, w, w1, w2, name):
    x, w1, w2, y = f64(x), f64(w1), f64(w2), f64(y)
    ref = blk.experts(x, idx, w, w1, w2, name)
    H, F = x.shape[1], w2.shape[2]
    tol = np.zeros_like(ref)
    for t in range(x.shape[0]):
        for i in range(idx.shape[1]):
            e = int(idx[t, i])
            if e < 0:
                continue
            u = w1[e] @ x[t]
            du = (H / 16 + 16) * 2.0 ** -23 * (np.abs(w1[e]) @ np.abs(x[t]))
            h = np.abs(blk.act(name, u))
            dh = (2.0 ** -8 + 2.0 ** -16) * h + 2 * (np.abs(u[:F]) + 1) * (np.abs(u[F:]) + 1) * (du[:F] + du[F:])
            dh += 2.0 ** -17 * (1 + np.abs(u[:F])) * np.abs(u[F:])
            tol[t] += abs(w[t, i]) * (np.abs(w2[e]) @ dh + (F / 16 + 16) * 2.0 ** -23 * (np.abs(w2[e]) @ h))
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + tol * 1.01 + 2.0 ** -20 * np.abs(ref) + 1e-30)
    for t in range(x.shape[0]):
        if np.any(ref[t]):
            assert orc.rel_frobenius(y[t], ref[t]) <= TOL_BF16, t
        else:
            assert not y[t].any()


def _check_route(idx, w, x, router, k, renorm):
    idx, w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    x, router = f64(x), f64(router)
    _, _, logits = blk.route(x, router, k, renorm)
    err = (x.shape[1] / 16 + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(router).T)
    for t in range(x.shape[0]):
        assert len(set(idx[t])) == k and idx[t].min() >= 0 and idx[t].max() < router.shape[0]
        l, d = logits[t][idx[t]], err[t].max()
        assert np.all(l[:-1] >= l[1:] - 2 * d)
        rest = np.delete(logits[t], idx[t])
        assert rest.size == 0 or rest.max() <= l[-1] + 2 * d
        p = np.exp(logits[t] - logits[t].max())
        want = p[idx[t]] / (p[idx[t]].sum() if renorm else p.sum())
        assert np.all(np.abs(w[t] - want) <= want * (2 * d + 2.0 ** -20))
    return idx, w


SHAPES = [  # T, E, k, H, F
    (1, 4, 2, 64, 64), (1, 1, 1, 8, 8), (2, 8, 8, 256, 136), (3, 5, 2, 200, 72), (7, 64, 6, 512, 352),
    (13, 16, 4, 1032, 200), (16, 8, 2, 128, 1000), (17, 33, 3, 264, 128), (33, 8, 1, 2048, 64), (64, 64, 6, 256, 192),
    (100, 4, 3, 136, 520), (128, 16, 2, 512, 128), (128, 256, 8, 128, 64), (128, 20, 16, 72, 40),
]


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
@pytest.mark.parametrize("act,renorm", [("swiglu", True), ("geglu", False)])
def test_layer(T, E, k, H, F, act, renorm):
    x, router, w1, w2 = _layer(T, E, H, F, seed=T + E)
    st = _status()
    ws = torch.full((gl.moe_workspace_bytes(T, E, k, H, F),), 0xFF, dtype=torch.uint8, device="cuda")
    y, idx, w = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router, act=gl.ACTS[act], renorm=renorm, workspace=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    i, ww = _check_route(idx, w, x, router, k, renorm)
    _check_y(y, x, i, ww, w1, w2, act)
    # again, over the dirty workspace: the same bits
    again = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router, act=gl.ACTS[act], renorm=renorm, workspace=ws)
    assert torch.equal(y, again[0]) and torch.equal(idx, again[1]) and torch.equal(w, again[2])


@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 4096, 1792), (5, 16, 4, 2048, 1408), (40, 8, 2, 1024, 3584)])
def test_layer_of_real_widths(T, E, k, H, F):
    x, router, w1, w2 = _layer(T, E, H, F, seed=3)
    st = _status()
    y, idx, w = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router)
    i, ww = _check_route(idx, w, x, router, k, True)
    _check_y(y, x, i, ww, w1, w2, "swiglu")
    assert int(st.item()) == 0


@pytest.mark.parametrize("T", [1, 9, 128])
def test_given_routing_with_absent_choices(T):
    E, k, H, F = 12, 4, 192, 104
    x, _, w1, w2 = _layer(T, E, H, F, seed=T)
    rng = np.random.default_rng(T)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[rng.random((T, k)) < 0.3] = -1
    if T > 1:
        idx[1] = -1           # a token without experts
    w = rng.standard_normal((T, k)).astype(np.float32)
    st = _status()
    ti, tw = torch.tensor(idx).cuda(), torch.tensor(w).cuda()
    y, ri, rw = gl.gl_moe_tokens(x, w1, w2, k, st, topk_idx=ti, topk_w=tw)
    assert int(st.item()) == 0 and ri is ti and rw is tw
    assert np.array_equal(ti.cpu().numpy(), idx) and np.array_equal(tw.cpu().numpy(), w)
    _check_y(y, x, idx, w.astype(np.float64), w1, w2, "swiglu")


def test_no_token_has_an_expert_and_every_token_has_the_same():
    T, E, k, H, F = 128, 6, 2, 256, 264
    x, _, w1, w2 = _layer(T, E, H, F)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    none = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    st = _status()
    y, _, _ = gl.gl_moe_tokens(x, w1, w2, k, st, topk_idx=none, topk_w=w)
    assert not y.any()
    same = torch.tensor([[5, 2]], dtype=torch.int32).repeat(T, 1).cuda()
    y, _, _ = gl.gl_moe_tokens(x, w1, w2, k, st, topk_idx=same, topk_w=w)
    _check_y(y, x, same.cpu().numpy(), w.cpu().numpy().astype(np.float64), w1, w2, "swiglu")
    assert int(st.item()) == 0


@pytest.mark.parametrize("bad", [6, -2, 1 << 20, -(1 << 31), "twice"])
def test_bad_indices_are_reported_and_nothing_is_written(bad):
    T, E, k, H, F = 5, 6, 3, 128, 64
    x, _, w1, w2 = _layer(T, E, H, F)
    idx = torch.tensor([[0, 1, 2]] * T, dtype=torch.int32)
    idx[3] = torch.tensor([4, 0, 4] if bad == "twice" else [1, bad, 0], dtype=torch.int32)
    st, y = _status(), sentinel_like(T, H)
    gl.gl_moe_tokens(x, w1, w2, k, st, topk_idx=idx.cuda(), topk_w=torch.ones(T, k, device="cuda"), y=y)
    assert int(st.item()) == gl.GL_DEV_BAD_INDEX and untouched(y)


def test_a_set_status_word_writes_nothing():
    x, router, w1, w2 = _layer(3, 4, 64, 64)
    st, y = _status() + gl.GL_DEV_NEG_SPLIT, sentinel_like(3, 64)
    i, w = torch.full((3, 2), 7, dtype=torch.int32, device="cuda"), torch.full((3, 2), 7.0, device="cuda")
    gl.gl_moe_tokens(x, w1, w2, 2, st, router_w=router, y=y, topk_idx=i, topk_w=w)
    assert untouched(y) and (i == 7).all() and (w == 7).all() and int(st.item()) == gl.GL_DEV_NEG_SPLIT


def test_ties_go_to_the_lower_expert():
    T, E, k, H, F = 20, 70, 8, 64, 64
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-1, 2, (T, H), generator=g).to(BF).cuda()
    router = torch.randint(-1, 2, (E, H), generator=g).to(BF)
    router[10:40] = router[3]
    router[50] = 0
    _, _, w1, w2 = _layer(T, E, H, F)
    _, idx, _ = gl.gl_moe_tokens(x, w1, w2, k, _status(), router_w=router.cuda())
    want, _, _ = blk.route(f64(x), f64(router), k, True)
    assert np.array_equal(idx.cpu().numpy(), want)  # integer logits are exact


def test_nan_stays_with_its_token():
    T, E, k, H, F = 6, 8, 2, 128, 64
    x, router, w1, w2 = _layer(T, E, H, F)
    x[2, 5] = float("nan")
    st = _status()
    y, idx, w = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router)
    assert torch.isnan(w[2]).all() and torch.isnan(y[2]).all() and int(st.item()) == 0
    keep = [0, 1, 3, 4, 5]
    assert torch.isfinite(y[keep]).all()
    _check_y(y[keep], x[keep], idx[keep].cpu().numpy(), w[keep].cpu().numpy().astype(np.float64), w1, w2, "swiglu")
    assert (idx >= 0).all() and (idx < E).all()


def test_per_group_weights():
    T, E, k, H, F = 10, 120, 4, 256, 128
    x, router, w1, w2 = _layer(T, E, H, F)
    want = gl.gl_moe_tokens(x, w1, w2, k, _status(), router_w=router)[0]
    l1, l2 = [w1[e].clone() for e in range(E)], [w2[e].clone() for e in range(E)]
    for a, b in ((l1, l2), (w1, l2), (l1, w2)):
        assert torch.equal(gl.gl_moe_tokens(x, a, b, k, _status(), router_w=router)[0], want)


def test_same_as_the_grouped_products():
    """The few-token layer and the same tokens through gl_fwd_act, sorted by expert."""
    T, E, k, H, F = 96, 8, 2, 512, 256
    x, router, w1, w2 = _layer(T, E, H, F)
    y, idx, w = gl.gl_moe_tokens(x, w1, w2, k, _status(), router_w=router)
    flat = torch.argsort(idx.reshape(-1).long(), stable=True)
    off, st = gl.gl_offsets(torch.bincount(idx.reshape(-1).long(), minlength=E), T * k)
    h, _ = gl.gl_fwd_act(x[flat // k], w1, None, off, st, gl.GL_ACT_SWIGLU)
    o, _ = gl.gl_fwd_act(h, w2, None, off, st, gl.GL_ACT_NONE)
    ref = torch.zeros(T, H, device="cuda").index_add_(0, flat // k, o.float() * w.reshape(-1)[flat, None])
    assert orc.rel_frobenius(f64(y), ref.double().cpu().numpy()) <= TOL_BF16


def test_timeouts_are_reported():
    x, router, w1, w2 = _layer(3, 4, 128, 64)
    st, y = _status(), sentinel_like(3, 128)
    gl.gl_moe_tokens(x, w1, w2, 2, st, router_w=router, y=y, wait_limit_us=2000, opt_flags=gl.GL_OPT_HOLD_LOADS)
    torch.cuda.synchronize()
    assert int(st.item()) == gl.GL_DEV_TIMEOUT and untouched(y)
    st.zero_()
    want = gl.gl_moe_tokens(x, w1, w2, 2, st, router_w=router, y=y)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and not untouched(y) and torch.isfinite(want[0]).all()


def test_captured_and_replayed_and_two_streams():
    T, E, k, H, F = 4, 16, 4, 512, 256
    x, router, w1, w2 = _layer(T, E, H, F)
    st = _status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router)
        b = gl.gl_moe_tokens(a[0], w1, w2, k, st, router_w=router)
    for seed in (5, 6):
        x.copy_(_rand(T, H, seed=seed))
        graph.replay()
        want = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router)
        want2 = gl.gl_moe_tokens(want[0], w1, w2, k, st, router_w=router)
        assert torch.equal(a[0], want[0]) and torch.equal(b[0], want2[0]) and torch.equal(b[1], want2[1])
    # two calls at once, each with its own workspace
    x2 = _rand(T, H, seed=11)
    torch.cuda.synchronize()
    outs = []
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s, v in ((s1, x), (s2, x2)):
        with torch.cuda.stream(s):
            for _ in range(5):
                outs.append(gl.gl_moe_tokens(v, w1, w2, k, st, router_w=router)[0])
    torch.cuda.synchronize()
    for v, got in ((x, outs[:5]), (x2, outs[5:])):
        want = gl.gl_moe_tokens(v, w1, w2, k, st, router_w=router)[0]
        assert all(torch.equal(want, o) for o in got)
    assert int(st.item()) == 0


def test_decoding_steps_of_two_blocks():
    """Norm with the residual's addition -> router and experts, twice, captured as a decoding step and replayed,
    against the oracle (which follows the experts that the call reports, up to near ties of bf16 inputs)."""
    T, E, k, H, F = 3, 16, 4, 256, 192
    layers = [(_rand(H, seed=i, std=0.1) + 1, _layer(T, E, H, F, seed=10 * i)[1:]) for i in (1, 2)]
    x, st = _rand(T, H, seed=5), _status()
    zero = torch.zeros_like(x)

    def step():
        add, res, kept = zero, x, []
        for gamma, (router, w1, w2) in layers:
            n = gl.gl_rmsnorm(add, gamma, 1e-5, residual=res)
            add, idx, w = gl.gl_moe_tokens(n["y"], w1, w2, k, st, router_w=router)
            res = n["sum"]
            kept.append((n["y"], idx, w, add))
        return kept, gl.gl_rmsnorm(add, layers[0][0], 1e-5, residual=res)["sum"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, out = step()
    for seed in (21, 22):
        x.copy_(_rand(T, H, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        stream = f64(x)
        for (gamma, (router, w1, w2)), (n, idx, w, y) in zip(layers, kept):
            _, _, norm = blk.rmsnorm(stream, None, f64(gamma), 1e-5)
            assert orc.rel_frobenius(f64(n), norm) <= TOL_BF16
            i, ww = _check_route(idx, w, n, router, k, True)
            _check_y(y, n, i, ww, w1, w2, "swiglu")
            stream = stream + blk.experts(norm, i, ww, f64(w1), f64(w2), "swiglu")
        assert orc.rel_frobenius(f64(out), stream) <= 1e-2


def test_beside_other_kernels_on_other_streams():
    """The cooperative kernel among products and norms of another stream and of another host thread."""
    import threading

    T, E, k, H, F = 5, 16, 4, 1024, 512
    x, router, w1, w2 = _layer(T, E, H, F)
    M, G = 4096, 8
    a, w, gamma = _rand(M, H, seed=1), _rand(G, 2048, H, seed=2, std=0.03), _rand(H, seed=3, std=0.1) + 1
    off, st = gl.gl_offsets(torch.full((G,), M // G, device="cuda"), M)
    st2 = _status()
    want = gl.gl_moe_tokens(x, w1, w2, k, st2, router_w=router)[0]
    want_y = gl.gl_fwd_act(a, w, None, off, st, gl.GL_ACT_SWIGLU)[0]
    want_n = gl.gl_rmsnorm(a, gamma, 1e-5)["y"]
    torch.cuda.synchronize()
    got, failed = {}, []

    def work(name, f):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[name] = [f() for _ in range(20)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # pragma: no cover
            failed.append((name, e))

    jobs = {"moe": lambda: gl.gl_moe_tokens(x, w1, w2, k, st2, router_w=router)[0],
            "act": lambda: gl.gl_fwd_act(a, w, None, off, st, gl.GL_ACT_SWIGLU)[0],
            "norm": lambda: gl.gl_rmsnorm(a, gamma, 1e-5)["y"]}
    threads = [threading.Thread(target=work, args=j) for j in jobs.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert int(st.item()) == 0 and int(st2.item()) == 0
    assert all(torch.equal(v, want) for v in got["moe"])
    assert all(torch.equal(v, want_y) for v in got["act"])
    assert all(torch.equal(v, want_n) for v in got["norm"])


@pytest.mark.parametrize("T", [1, 2, 3, 9, 128])
def test_weights_of_absent_choices_are_not_used(T):
    """NaN and infinite weights at index -1: the bits that zeros there give, and zeros for a token without experts."""
    E, k, H, F = 12, 4, 192, 104
    x, _, w1, w2 = _layer(T, E, H, F, seed=T)
    rng = np.random.default_rng(T)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[rng.random((T, k)) < 0.4] = -1
    idx[0] = [-1, 3, -1, 7]  # every token count has a token that drops some of its choices
    if T > 1:
        idx[1] = -1
    w = rng.standard_normal((T, k)).astype(np.float32)
    ti = torch.tensor(idx).cuda()
    want = gl.gl_moe_tokens(x, w1, w2, k, _status(), topk_idx=ti, topk_w=torch.tensor(np.where(idx < 0, 0, w)).cuda())[0]
    _check_y(want, x, idx, w.astype(np.float64), w1, w2, "swiglu")
    for v in (np.nan, np.inf, -np.inf):
        st = _status()
        tw = torch.tensor(np.where(idx < 0, np.float32(v), w)).cuda()
        y = gl.gl_moe_tokens(x, w1, w2, k, st, topk_idx=ti, topk_w=tw)[0]
        assert torch.equal(y, want) and int(st.item()) == 0
        if T > 1:
            assert not y[1].any()


@pytest.mark.parametrize("T,given", [(3, False), (3, True), (40, False), (40, True)])
def test_a_status_word_that_changes_meanwhile(T, given):
    """Another stream sets and clears the status word while calls run: each call writes all of its outputs or none of
    them, and none waits for CTAs that went by another value (such a wait takes two seconds)."""
    E, k, H, F, n = 16, 4, 512, 256, 80
    x, router, w1, w2 = _layer(T, E, H, F)
    st, ws = _status(), torch.empty(gl.moe_workspace_bytes(T, E, k, H, F), dtype=torch.uint8, device="cuda")
    want = gl.gl_moe_tokens(x, w1, w2, k, st, router_w=router, workspace=ws)
    ys = [sentinel_like(T, H) for _ in range(n)]
    if given:
        routes = [dict(topk_idx=want[1], topk_w=want[2])] * n
    else:
        routes = [dict(router_w=router, topk_idx=torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
                       topk_w=torch.full((T, k), -7.0, device="cuda")) for _ in range(n)]
    calls, setter = torch.cuda.Stream(), torch.cuda.Stream()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record(calls)
    for y, r in zip(ys, routes):
        with torch.cuda.stream(calls):
            gl.gl_moe_tokens(x, w1, w2, k, st, y=y, workspace=ws, **r)
        with torch.cuda.stream(setter):
            for _ in range(4):
                st.fill_(gl.GL_DEV_NEG_SPLIT)
                st.zero_()
    end.record(calls)
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) < 1500
    for y, r in zip(ys, routes):
        if untouched(y):
            assert given or ((r["topk_idx"] == -7).all() and (r["topk_w"] == -7).all())
        else:
            assert torch.equal(y, want[0]) and torch.equal(r["topk_idx"], want[1]) and torch.equal(r["topk_w"], want[2])
    st.zero_()
    assert torch.equal(gl.gl_moe_tokens(x, w1, w2, k, st, workspace=ws, **routes[0])[0], want[0]) and int(st.item()) == 0
