"""The training operators together: a MoE layer's gradients through the library against torch's
autograd in float64, and losses that fall, with fp32 and with 8-bit optimizer states."""

import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.gpu_helpers import host, say              # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "moe_train_step", os.path.join(ROOT, "examples", "moe_train_step.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["moe_train_step"] = m
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(example):
    """The reference is the dense layer in float64 on the same bf16 weights and inputs, with the
    library's selection.  Between them lie bf16 roundings of rows and outputs (2^-8 of values
    that then meet in sums of random sign): relative errors in the 2-norm of a few 2^-8, 3 %
    allowed."""
    say("case: train step, gradients")
    geo = example.Geometry(R=2, T=64, K=2, E=4, S=1, H=64, F=32, q_min=4)
    layer = example.Layer(geo, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(2, 64, 64, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(2, 64, 64, generator=gen, device="cuda").to(torch.bfloat16)
    y, saved = layer.forward(x)
    ids, plan = saved[2], saved[4]
    assert int((plan["slot_expert"] >= 0).sum()) > 0                 # replicas were used
    ids, y = ids.cpu().long(), y.double().cpu()
    dx = layer.backward(dy, saved)
    assert int(host(layer.err)[0]) == 0

    xd = x.double().cpu().requires_grad_()
    wr = layer.router.double().cpu().requires_grad_()
    we = layer.main_w.double().cpu().requires_grad_()
    logits = xd @ wr + layer.lean.double().cpu()
    w = torch.softmax(logits.gather(-1, ids), -1)                    # renormalised softmax
    want = torch.zeros_like(xd)
    for e in range(geo.E):
        a, b, c = we[e].view(3, -1)
        h = (torch.nn.functional.silu(xd @ a.view(64, 32)) * (xd @ b.view(64, 32))) @ c.view(32, 64)
        want = want + h * (w * (ids == e)).sum(-1, keepdim=True)
    (want * dy.double().cpu()).sum().backward()

    def near(got, ref, name):
        err = float((got.double().cpu() - ref).norm() / ref.norm())
        say(f"{name}: relative error {err:.2e}")
        assert err < 0.03, name

    near(y, want.detach(), "y")
    near(layer.main_grad, we.grad, "experts")
    near(layer.router_grad, wr.grad, "router")
    near(dx, xd.grad, "x")


@pytest.mark.parametrize("state_bits", [32, 8])
def test_losses_fall(example, state_bits):
    say("case: train step, losses", state_bits)
    losses = example.train(steps=40, seed=0, state_bits=state_bits)
    assert np.isfinite(losses).all()
    assert losses[-1] < 0.6 * losses[0]
    again = example.train(steps=3, seed=0, state_bits=state_bits)
    assert again[0] == losses[0]
