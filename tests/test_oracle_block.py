"""The block oracle (norm, activations, few-token layer) against torch autograd
in 64 bits, differences, and values worked by hand."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as blk


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_is_the_autograd_of_its_formula(residual):
    rng = np.random.default_rng(5)
    x, r, dy, ds = (torch.tensor(rng.standard_normal((7, 40)), requires_grad=True) for _ in range(4))
    gamma = torch.tensor(rng.standard_normal(40), requires_grad=True)
    s = x + r if residual else x
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-3) * gamma
    (y * dy.detach() + s * ds.detach()).sum().backward()
    n = [t.detach().numpy() for t in (x, r, gamma, dy, ds)]
    s64, rstd, y64 = blk.rmsnorm(n[0], n[1] if residual else None, n[2], 1e-3)
    np.testing.assert_allclose(y64, y.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(s64, s.detach().numpy(), rtol=1e-12)
    dx, dgamma = blk.rmsnorm_bwd(n[3], s64, n[2], rstd, n[4])
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(dgamma, gamma.grad.numpy(), rtol=1e-9, atol=1e-12)
    if residual:
        np.testing.assert_allclose(dx, r.grad.numpy(), rtol=1e-9, atol=1e-12)


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(6)
    x, dy = rng.standard_normal((3, 16)), rng.standard_normal((3, 16))
    gamma = rng.standard_normal(16)

    def loss(x, gamma):
        return float(np.sum(blk.rmsnorm(x, None, gamma, 1e-5)[2] * dy))

    s, rstd, _ = blk.rmsnorm(x, None, gamma, 1e-5)
    dx, dgamma = blk.rmsnorm_bwd(dy, s, gamma, rstd, None)
    h = 1e-6
    for i, j in ((0, 0), (1, 7), (2, 15)):
        e = np.zeros_like(x)
        e[i, j] = h
        assert abs((loss(x + e, gamma) - loss(x - e, gamma)) / (2 * h) - dx[i, j]) < 1e-7
        assert abs((loss(x, gamma + e[i]) - loss(x, gamma - e[i])) / (2 * h) - dgamma[j]) < 1e-7


def test_rmsnorm_by_hand():
    s, rstd, y = blk.rmsnorm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    assert rstd[0] == pytest.approx(1 / np.sqrt(12.5))
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])


def _torch_act(name, u):
    F = torch.nn.functional
    half = u.shape[-1] // 2
    return {"none": lambda: u, "relu": lambda: F.relu(u), "relu2": lambda: F.relu(u) ** 2,
            "gelu": lambda: F.gelu(u, approximate="tanh"), "silu": lambda: F.silu(u),
            "swiglu": lambda: F.silu(u[..., :half]) * u[..., half:],
            "geglu": lambda: F.gelu(u[..., :half], approximate="tanh") * u[..., half:]}[name]()


@pytest.mark.parametrize("name", blk.ACTS)
def test_activation_and_its_gradient_against_autograd(name):
    rng = np.random.default_rng(3)
    u = torch.tensor(rng.standard_normal((9, 24)) * 4, requires_grad=True)
    y = _torch_act(name, u)
    dy = torch.tensor(rng.standard_normal(y.shape))
    (y * dy).sum().backward()
    np.testing.assert_allclose(blk.act(name, u.detach().numpy()), y.detach().numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(blk.act_bwd(name, u.detach().numpy(), dy.numpy()), u.grad.numpy(), rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("name", blk.ACTS[1:])
def test_activation_gradient_against_differences(name):
    rng = np.random.default_rng(8)
    z, w = rng.standard_normal((4, 12)) * 2, rng.standard_normal((1, 5, 12 // (2 if name in blk.GATED else 1)))
    dy = rng.standard_normal((4, 5))

    def loss(z):
        return float(np.sum(blk.fwd_act(blk.act(name, z), w, None, [4], "none", None)[0] * dy))

    dz, h = blk.dgrad_act(dy, w, [4], name, z), 1e-6
    for i, j in ((0, 0), (1, 5), (2, 6), (3, 11)):
        e = np.zeros_like(z)
        e[i, j] = h
        assert abs((loss(z + e) - loss(z - e)) / (2 * h) - dz[i, j]) < 1e-6 * (1 + abs(dz[i, j]))


@pytest.mark.parametrize("name", blk.ACTS[1:])
def test_grouped_products_with_activations_against_autograd(name):
    rng = np.random.default_rng(4)
    m = [5, 0, 3]
    two = 2 if name in blk.GATED else 1
    x = torch.tensor(rng.standard_normal((8, 6)))
    z = torch.tensor(rng.standard_normal((8, 10 * two)), requires_grad=True)
    w = torch.tensor(rng.standard_normal((3, 4, 10)))
    dy, r = rng.standard_normal((8, 4)), rng.standard_normal((8, 4))
    h = _torch_act(name, z)
    y = torch.cat([h[a:b] @ w[g].T for g, (a, b) in enumerate(((0, 5), (5, 5), (5, 8)))]) + torch.tensor(r)
    (y * torch.tensor(dy)).sum().backward()
    np.testing.assert_allclose(blk.dgrad_act(dy, w.numpy(), m, name, z.detach().numpy()), z.grad.numpy(), rtol=1e-9,
                               atol=1e-12)
    got, u = blk.fwd_act(h.detach().numpy(), w.numpy(), None, m, "none", r)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-10)
    np.testing.assert_allclose(u + r, got, rtol=1e-12)


def test_routing_by_hand():
    x = np.array([[1.0, 0.0], [0.0, 2.0], [0.0, 0.0]])
    router = np.array([[0.0, 1.0], [1.0, 0.0], [0.0, 1.0], [np.log(2.0), 0.0]])
    idx, w, _ = blk.route(x, router, 2, True)
    assert idx.tolist() == [[1, 3], [0, 2], [0, 1]]  # ties: the lower expert
    e = np.e
    np.testing.assert_allclose(w, [[e / (e + 2), 2 / (e + 2)], [0.5, 0.5], [0.5, 0.5]])
    _, w, _ = blk.route(x, router, 2, False)
    np.testing.assert_allclose(w[0], [e / (e + 4), 2 / (e + 4)])


def test_experts_against_torch_and_the_grouped_products():
    rng = np.random.default_rng(9)
    T, E, k, H, F = 5, 4, 2, 6, 3
    x, w1, w2 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * F, H)), rng.standard_normal((E, H, F))
    idx, w, _ = blk.route(x, rng.standard_normal((E, H)), k, True)
    y = blk.experts(x, idx, w, w1, w2, "swiglu")
    want = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for i in range(k):
            u = torch.tensor(w1[idx[t, i]]) @ torch.tensor(x[t])
            want[t] += w[t, i] * (torch.tensor(w2[idx[t, i]]) @ (torch.nn.functional.silu(u[:F]) * u[F:]))
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-10)
    # the same layer as the grouped products over rows sorted by expert
    flat = np.argsort(idx.reshape(-1), kind="stable")
    m = [int((idx == e).sum()) for e in range(E)]
    h, _ = blk.fwd_act(x[flat // k], w1, None, m, "swiglu", None)
    o, _ = blk.fwd_act(h, w2, None, m, "none", None)
    grouped = np.zeros((T, H))
    np.add.at(grouped, flat // k, o * w.reshape(-1)[flat, None])
    np.testing.assert_allclose(y, grouped, rtol=1e-10)
    idx[2] = -1
    assert not blk.experts(x, idx, w, w1, w2, "swiglu")[2].any()
