"""The balance loss and the 8-bit expert path inside the example's layer: gradients with the
balance loss against torch's autograd in float64, outputs in 8 bits against the same steps in
float64."""

import importlib.util
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle as O                                       # noqa: E402
from tests.gpu_helpers import host, say                  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "moe_train_step_int8", os.path.join(ROOT, "examples", "moe_train_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["moe_train_step_int8"] = m
    spec.loader.exec_module(m)
    return m


def batch(seed, R, T, H):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(R, T, H, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]


def test_router_gradient_with_the_balance_loss(example):
    """The balance loss reaches the router and x alone; the library's selection is taken over.  The
    difference between two backward passes, with and without it, against autograd: logits and
    gradients are fp32, so what is left are fp32 sums over 128 tokens of gradients whose parts
    cancel, and the difference of two gradients of the task, 2^-24 of which a thousand steps of
    rounding make 1e-4 of a balance gradient that the weight makes about as large."""
    say("case: layer, balance gradient")
    geo = example.Geometry(R=2, T=64, K=2, E=4, S=1, H=64, F=32, q_min=4, balance=500.0)
    layer = example.Layer(geo, seed=3)
    x, dy = batch(4, 2, 64, 64)
    grads = []
    for weight in (500.0, 0.0):
        geo.balance = weight
        y, saved = layer.forward(x)
        layer.backward(dy, saved)
        grads.append(layer.router_grad.double().cpu().clone())
    assert int(host(layer.err)[0]) == 0
    ids, logits = saved[2].cpu().long(), saved[1]
    wr = layer.router.double().cpu().requires_grad_()
    z = x.double().cpu() @ wr + layer.lean.double().cpu()
    p = torch.softmax(z, -1)
    counts = torch.stack([torch.bincount(i.reshape(-1), minlength=4) for i in ids]).double()
    loss = (counts * p.mean(1)).sum(-1) * 4 / (2 * 64)
    (500.0 * loss.mean()).backward()
    got = layer.balance_loss(logits, saved[2])[0]
    assert torch.allclose(got.double().cpu(), loss.detach(), rtol=1e-5)
    err = float((grads[0] - grads[1] - wr.grad).norm() / wr.grad.norm())
    size = float(grads[1].norm() / wr.grad.norm())
    say(f"relative error {err:.2e}, task gradient {size:.1f} times as large")
    assert err < 1e-4 * max(1.0, size)


@pytest.mark.parametrize("R,T,K,E,S,H,F", [(2, 64, 2, 4, 1, 64, 32), (4, 100, 3, 8, 2, 128, 48),
                                           (1, 1, 2, 4, 0, 64, 16), (2, 1000, 2, 4, 1, 256, 128)])
def test_outputs_in_8_bits(example, R, T, K, E, S, H, F):
    """The same steps in float64 on the library's routing and plan: rows and weights to integers by
    their definition, exact products, the middle rounded to bf16 and to integers again.  A middle
    value within an fp32 rounding of a bf16 border may take the other side, and shift its row's
    integers by a step where it is the largest: 2^-8 of it, and single integers otherwise.  The
    outputs are rounded twice to bf16 (product and combine, 2^-8 each at most): 2 * 2^-8 in the
    2-norm, and as much again for the shifted integers."""
    say("case: layer in 8 bits", R, T, K, E, S, H, F)
    geo = example.Geometry(R=R, T=T, K=K, E=E, S=S, H=H, F=F, q_min=4)
    layer = example.Layer(geo, seed=5)
    layer.quantise()
    x, _ = batch(6, R, T, H)
    y = layer.forward_int8(x)
    _, (_, _, ids, w, plan, *_) = layer.forward(x)
    assert int(host(layer.err)[0]) == 0
    if S and T >= 64:
        assert int((plan["slot_expert"] >= 0).sum()) > 0
    q, scale = O.quant_rows(x.double().cpu().numpy())
    out = np.zeros((R, T, H))
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    mats = [[m.double().cpu().numpy() for m in layer._matrices(m)] for m in layer.main_w]
    for e in range(E):
        gate, up, down = mats[e]
        w1, s1 = O.quant_rows(np.concatenate([gate.T, up.T]))
        w2, s2 = O.quant_rows(down.T)
        r, t, k = np.nonzero(ids == e)
        if not len(r):
            continue
        z = (q[r, t].astype(float) @ w1.T.astype(float)) * s1 * scale[r, t][:, None].astype(float)
        a, b = np.split(z, 2, axis=-1)
        h = torch.from_numpy(a / (1 + np.exp(-a)) * b).to(torch.bfloat16).double().numpy()
        qh, sh = O.quant_rows(h)
        z = (qh.astype(float) @ w2.T.astype(float)) * s2 * sh[:, None].astype(float)
        np.add.at(out, (r, t), z * w[r, t, k][:, None])
    err = float(np.linalg.norm(y.double().cpu().numpy() - out) / np.linalg.norm(out))
    say(f"relative error {err:.2e}")
    assert err < 4 * 2.0 ** -8


def test_the_example_runs(example, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["moe_train_step.py", "--steps", "3", "--balance", "0.01"])
    example.main()
    assert "balance" in capsys.readouterr().out
