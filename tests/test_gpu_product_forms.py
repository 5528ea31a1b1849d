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
from tests.test_gpu_int8 import operands, blocks, run_product, check_product   # noqa: E402

pytestmark = pytest.mark.gpu


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
