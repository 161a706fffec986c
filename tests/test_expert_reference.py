"""CPU: the 64-bit references that the experts' GPU tests hold the kernels to --
their gradients against central differences of their forward pass."""
import pytest
import torch

import expert_reference as ref


def f64(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("name", ["none", "silu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("glu", [True, False])
def test_gradients_are_the_differences(glu, name):
    m, k, f = 5, 7, 4
    n = 2 * f if glu else f
    x, w, b, c = f64(m, k, seed=1), f64(n, k, seed=2), f64(n, seed=3), f64(m, f, seed=4)

    def loss(x, w, b):
        return (c * ref.forward(x, w, b, glu, name)[1]).sum()

    z = ref.forward(x, w, b, glu, name)[0]
    assert (z.abs() > 1e-3).all()  # away from relu's corner
    dz, _ = ref.grad(c, z, glu, name)
    grads = {"x": dz @ w, "w": dz.T @ x, "b": dz.sum(0)}
    values, h = {"x": x, "w": w, "b": b}, 1e-5
    for key, v in values.items():
        for i in range(v.numel()):
            up, down = v.clone().view(-1), v.clone().view(-1)
            up[i] += h
            down[i] -= h
            num = (loss(**{**values, key: up.view(v.shape)}) - loss(**{**values, key: down.view(v.shape)})) / (2 * h)
            # central difference: h^2 third derivatives, and 1e-16 / h of rounding
            assert abs(num - grads[key].reshape(-1)[i]) < 1e-7 * (1 + abs(num))


@pytest.mark.parametrize("name", ["silu", "gelu_tanh", "relu"])
def test_activations_at_the_ends(name):
    z = torch.tensor([-1e30, -30.0, -0.0, 0.0, 30.0, 1e30], dtype=torch.float64)
    a, s = ref.act(z, name), ref.slope(z, name)
    assert torch.equal(a[[4, 5]], z[[4, 5]]) or torch.allclose(a[[4, 5]], z[[4, 5]])
    assert torch.all(a[:4].abs() < 1e-9)
    assert torch.allclose(s[[1, 4]], torch.tensor([0.0, 1.0], dtype=torch.float64), atol=1e-9)
