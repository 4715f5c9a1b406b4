"""The example's feed-forward block serves the weights that it has: its host
logic on the CPU, with the library's calls replaced by plain products."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Plain:
    """The calls that decode() and serve() make, unquantized; `laid_out` counts the weights that are laid out."""

    def __init__(self):
        self.laid_out = 0

    def mxfp4_fp8_quantize_pair(self, gate, up, axis=1):
        self.laid_out += 1
        return gate.detach().clone(), up.detach().clone()

    def mxfp4_fp8_quantize(self, x, axis=1, block_rows=1):
        self.laid_out += 1
        return x.detach().clone()

    def mxfp4_fp8_rmsnorm(self, x, weight, eps, residual=None, sum_out=None):
        r = sum_out.copy_(x + residual)
        f = r.float()
        return f * torch.rsqrt(f.square().mean(1, keepdim=True) + eps) * weight.float(), r

    def mxfp4_fp8_gated(self, q, pair, act="silu"):
        g, u = (q @ w.float().t() for w in pair)
        return g * torch.sigmoid(g) * u

    def mxfp4_fp8_gemm(self, a, b):
        return (a @ b.float().t()).to(torch.bfloat16)


@pytest.fixture()
def example(monkeypatch):
    spec = importlib.util.spec_from_file_location("fp8_feed_forward_cpu",
                                                  os.path.join(ROOT, "examples", "fp8_feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "mx", Plain())
    return m


def case(example):
    block = example.FeedForward(64, 96, device="cpu", seed=2)
    gen = torch.Generator().manual_seed(3)
    x, res = (torch.randn((5, 64), generator=gen).to(torch.bfloat16) for _ in range(2))
    fresh = lambda: example.FeedForward.decode(copy(example, block), x, res.clone())[0]  # noqa: E731
    return block, x, res, fresh


def copy(example, block):
    """A block that has the same weights and has served nothing yet."""
    other = example.FeedForward(64, 96, device="cpu", seed=7)
    with torch.no_grad():
        for a, b in zip(other.parameters(), block.parameters()):
            a.copy_(b)
    return other


def change_in_place(block):
    with torch.no_grad():
        for p in block.parameters():
            p.mul_(1.5)


def change_data(block):
    for p in block.parameters():   # (leaves the tensors' versions as they are)
        p.data.mul_(-0.5)


def change_optimizer(block):
    for p in block.parameters():
        p.grad = torch.ones_like(p)
    torch.optim.SGD(block.parameters(), lr=0.125).step()


def change_objects(block):
    block.gate, block.up = block.up, block.gate


@pytest.mark.parametrize("change", [change_in_place, change_data, change_optimizer, change_objects])
def test_decode_sees_every_change_of_a_weight(example, change):
    block, x, res, fresh = case(example)
    before = block.decode(x, res.clone())[0]
    assert torch.equal(before, fresh())
    change(block)
    after = block.decode(x, res.clone())[0]
    assert torch.equal(after, fresh())
    assert not torch.equal(after, before)


def test_served_weights_are_laid_out_once(example):
    """serve() lays the weights out as they are; decode() with them lays out nothing."""
    block, x, res, _ = case(example)
    served = block.serve()
    n = example.mx.laid_out
    before = block.decode(x, res.clone())[0]
    assert example.mx.laid_out > n
    n = example.mx.laid_out
    for _ in range(3):
        assert torch.equal(block.decode(x, res.clone(), served)[0], before)
    assert example.mx.laid_out == n
    change_in_place(block)
    with torch.no_grad():
        block.norm.mul_(1 / 1.5)   # (read by every call: only the products' weights are laid out)
    assert torch.equal(block.decode(x, res.clone(), served)[0], before)
    assert torch.equal(block.decode(x, res.clone(), block.serve())[0], block.decode(x, res.clone())[0])
