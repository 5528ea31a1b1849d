"""GPU parity of every form of the experts' product over a plan with replica slots.  Tolerances are
those of test_gpu_int8: three fp32 roundings (SwiGLU (4 |gate| + 16) of 2^-24) and the store."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, host, say, err_word   # noqa: E402
from tests.product_shapes import SHAPES                  # noqa: E402
from tests.rules import form                             # noqa: E402
from tests.test_gpu_int8 import operands, blocks, run_product, check_product   # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.mark.parametrize("act", [U.PRODUCT_PLAIN, U.PRODUCT_SWIGLU])
@pytest.mark.parametrize("even", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_form(shape, even, act):
    say("case: product form", *shape, even, act)
    rows, R, E, S, N, D, *_ = shape
    o = operands(rows, R, E, S, N, D, rows + N + D)
    off = blocks(np.random.default_rng(rows + N), rows, R * (E // R + S), 2, 3, even)
    n_out = N // 2 if act == U.PRODUCT_SWIGLU else N
    out = torch.full((rows, n_out), 7.0, dtype=torch.bfloat16, device=DEV)
    err = err_word()
    run_product(o, off, R, S, act, out, err)
    assert int(host(err)[0]) == 0
    check_product(o, off, R, E, S, act, out, 7.0)
    again = torch.full_like(out, 7.0)
    run_product(o, off, R, S, act, again)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("rows", [7, 60, 3000])
def test_gates_far_below_zero(rows):
    """silu(g) = g / (1 + e^-g) where e^-g passes what a float holds: still a number, of which a
    large up value makes an ordinary one.  In units of 2^-24 the gate is off by 3, the two halves of
    its exponential by (1.5 |gate| + 4) with what the gate's own makes (3 |gate|), the reciprocal, four
    products and the up value by 10: within (5 |gate| + 20), then the store."""
    say("case: product, gates far below zero", rows)
    n, D = 520, 48
    assert rows < 100 or form(rows, 1, n, D, True) == "large"
    gate = np.linspace(-170, 2, n).astype(np.float32)
    up = np.float32(10.0) ** np.linspace(0, 37, 13)
    up = np.resize(up, n).astype(np.float32)
    q = torch.ones(rows, D, dtype=torch.int8, device=DEV)
    w = torch.ones(1, 2 * n, D, dtype=torch.int8, device=DEV)
    ws = torch.from_numpy(np.concatenate([gate, up]) / np.float32(D)).to(DEV)[None]
    qs = torch.linspace(0.9, 1.0, rows, device=DEV)
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    U.expert_product(q, qs, w, ws, act=U.PRODUCT_SWIGLU, out=out)
    z = D * host(ws).astype(np.float64) * host(qs).astype(np.float64)[:, None]
    g, u = z[:, :n], z[:, n:]
    y = g / (1 + np.exp(-g)) * u
    got = out.double().cpu().numpy()
    room = (5 * np.abs(g) + 20) * EPS * np.abs(y)
    assert (np.abs(got - y) <= room + 2.0 ** -8 * (np.abs(y) + room) + 2.0 ** -133).all()
    assert (got[(np.abs(y) > 2.0 ** -126)] != 0).all()
