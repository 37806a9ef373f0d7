"""The example that runs the operators together: its gradients against the formulas' in 64 bits
without any 8-bit checkpoint, and a training run."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_sharded_mixed_02_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_blocks.py")
    spec = importlib.util.spec_from_file_location("residual_blocks", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return torch, module


def plain(torch, net, h):
    """The same stack in 64 bits; (weights by name, h0, the last boundary's rows)."""
    w = {name: net.weight(name).double().requires_grad_() for name in net.place}
    h0 = h.double().requires_grad_()
    r, y = h0, None
    for i in range(net.blocks + 1):
        if i:
            yh = y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-5)
            r = r + w[f"gate{i}"] * (w[f"post_w{i}"] * yh)
        mean = r.mean(1, keepdim=True)
        xh = (r - mean) * torch.rsqrt((r - mean).square().mean(1, keepdim=True) + 1e-5)
        x = w[f"pre_w{i}"] * xh + w[f"pre_b{i}"]
        if i < net.blocks:
            y = torch.tanh(x @ w[f"w1_{i}"].T + w[f"b1_{i}"]) @ w[f"w2_{i}"].T + w[f"b2_{i}"]
    return w, h0, x


@pytest.mark.parametrize("d,f,blocks,tokens", [(64, 256, 2, 300), (100, 36, 1, 77)])
def test_gradients_of_the_stack(example, d, f, blocks, tokens):
    torch, module = example
    net = module.ResidualBlocks(d, f, blocks, tokens, ranks=1)
    torch.manual_seed(1)
    for name in net.place:                                   # weights and biases away from 1 and 0
        if len(net.place[name][1]) == 1:
            net.weight(name).add_(0.2 * torch.randn(net.place[name][1], device="cuda").half())
    h, dx = torch.randn(tokens, d, device="cuda"), torch.randn(tokens, d, device="cuda").half()
    w, h0, want = plain(torch, net, h)
    want.backward(dx.double())
    got = net.forward(h.clone())
    # roundings to 16 bits, a few in each block
    want = want.detach()
    assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8
    dh = net.backward(dx, 0)
    # a block of 32 codes has steps of at most max/64, about 0.04 of its values' rms: an error of
    # 0.01 of it in each checkpoint, some of which add up over the blocks
    assert float((dh.double() - h0.grad).norm() / h0.grad.norm()) < 2.0 ** -5
    for name in net.place:
        g = net.grad(0, name).double()
        assert float((g - w[name].grad).norm() / w[name].grad.norm()) < 2.0 ** -5, name
    net.close()


def test_training_lowers_the_loss(example):
    torch, module = example
    losses, kept = module.train(steps=40, d=128, f=256, blocks=2, tokens=300)
    assert all(l == l and l < 10 for l in losses)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])
    again, _ = module.train(steps=3, d=128, f=256, blocks=2, tokens=300)
    assert again == losses[:3]                                                 # sums in a fixed order: the same run twice
    # 8 bits and a 32nd for each value, 16 bytes a row and boundary
    assert kept <= 300 * ((3 + 2) * (128 + 32) + 2 * (256 + 32) + 3 * 16)
