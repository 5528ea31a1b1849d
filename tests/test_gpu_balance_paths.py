"""The balance loss and its gradient where a call's blocks do more than one thing: many chunks of a
sequence, which several blocks join, and chunks of more than one pass over the lanes of a block.

Every case asks the library's own arithmetic whether it is there for what it is there for.
Tolerances in eps = 2^-24: a score is within (4 spread + 160) eps, spread the largest logit or
distance to a row's largest; a lane adds its chunk's passes in a row, then at most six butterflies and four
waves, all of positive numbers; chunks are joined in 64 bits.  The gradient's are those of
test_gpu_balance_range."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle as O                                       # noqa: E402
from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, to_dev, host, say, err_word   # noqa: E402
from tests.rules import chunk as chunk_tokens, sliced   # noqa: E402
from tests.test_gpu_balance_range import EPS, spread, oracle_and_room, check   # noqa: E402

pytestmark = pytest.mark.gpu


def make(seed, n, E, K, G, ragged, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(1, n, E, generator=g, device=DEV) * 2 +
         torch.randn(E, generator=g, device=DEV)).to(dtype)
    ids = torch.topk(x.float(), K, dim=-1).indices.to(torch.int32)
    ids[0, torch.rand(n, generator=g, device=DEV) < 0.1] = -1
    if not ragged:
        return x, ids, None
    rng = np.random.default_rng(seed)
    off = np.sort(rng.integers(0, n + 1, G + 1)).astype(np.int32)
    return x, ids, off


def check_forward(got, x, ids, G, off, score, passes):
    loss, counts, prob, tokens = (host(t) for t in got)
    want = O.balance_loss(x, ids, G, off, score)
    rel = (4 * spread(x, score) + 160 + passes + 10) * EPS
    assert np.array_equal(counts, want[1]) and np.array_equal(tokens, want[3])
    assert (np.abs(prob - want[2]) <= rel * want[2] + 2.0 ** -126).all()
    assert (np.abs(loss - want[0]) <= (rel + 4 * EPS) * want[0]).all()


# tokens, E, K, sequences, ragged, dtype, score
JOINED = [(13000, 128, 8, 1, False, torch.float32, 0), (8190, 200, 4, 2, True, torch.float32, 1),
          (25601, 128, 8, 2, True, torch.bfloat16, 1), (17001, 99, 3, 1, True, torch.bfloat16, 0),
          (3100, 1000, 8, 3, True, torch.bfloat16, 0), (1600, 4096, 6, 3, True, torch.bfloat16, 1),
          (68, 4096, 2, 1, False, torch.float32, 0), (30000, 512, 6, 4, False, torch.float32, 1)]


@pytest.mark.parametrize("case", JOINED)
def test_sequences_of_many_chunks(case):
    """So many chunks of so many experts that several blocks join a sequence, and a launch of its own
    adds their parts of the loss."""
    say("case: balance, joined by several blocks", *case)
    n, E, K, G, ragged, dtype, score = case
    size = 4 if dtype == torch.float32 else 2
    chunk, passes = chunk_tokens(n, E, size)
    chunks = n // chunk + G if ragged else G * -(-(n // G) // chunk)
    assert sliced(chunks // G, E), chunks // G
    x, ids, off = make(n, n, E, K, G, ragged, dtype)
    off_d, err = None if off is None else to_dev(off), err_word()
    got = U.balance_loss(x, ids, G, seq_offset=off_d, score=score, err=err)
    check_forward(got, x.double().cpu().numpy(), host(ids), G, off, score, passes)
    again = U.balance_loss(x, ids, G, seq_offset=off_d, score=score)
    assert all(torch.equal(a, b) for a, b in zip(got, again)) and int(host(err)[0]) == 0


# tokens, E, sequences, ragged, dtype, score
PASSES = [(17003, 1000, 1, False, torch.float32, 0), (33001, 520, 5, True, torch.bfloat16, 1),
          (16999, 1100, 3, True, torch.bfloat16, 0), (600011, 30, 4, True, torch.float32, 1),
          (150001, 100, 1, False, torch.bfloat16, 1), (300007, 3, 2, True, torch.float32, 0)]


@pytest.mark.parametrize("case", PASSES)
def test_chunks_of_several_passes(case):
    """So many tokens that a gradient block goes over its lanes more than once, the last time with
    tokens for some of them: a row, and a row of what the gradient is added to, are on their way
    while others are worked on, also where they lie in the output."""
    say("case: balance, several passes", *case)
    n, E, G, ragged, dtype, score = case
    size = 4 if dtype == torch.float32 else 2
    chunk, passes = chunk_tokens(n, E, size, grad=True)
    assert passes >= 2 and n % chunk != 0
    x, ids, off = make(n, n, E, 2, G, ragged, dtype)
    off_d, err = None if off is None else to_dev(off), err_word()
    args = dict(seq_offset=off_d, score=score, err=err)
    got = U.balance_loss(x, ids, G, **args)
    x64, ids_h = x.double().cpu().numpy(), host(ids)
    own_passes = chunk_tokens(n, E, size)[1]
    check_forward(got, x64, ids_h, G, off, score, own_passes)
    dloss = np.random.default_rng(E).normal(size=G).astype(np.float32)
    dl = to_dev(dloss, torch.float32)
    d = U.balance_loss_grad(dl, x, ids, got[1], got[3], **args)
    ref, room = oracle_and_room(dloss, x64, ids_h, host(got[1]), host(got[3]), G, off, score)
    check(d, ref, room, dtype)
    size_of = float(np.abs(ref).max())
    g = torch.Generator(device=DEV).manual_seed(1)
    base = (torch.randn(x.shape, generator=g, device=DEV) * size_of).to(dtype)
    both = U.balance_loss_grad(dl, x, ids, got[1], got[3], add=base, **args)
    total = base.double().cpu().numpy() + ref
    check(both, total, room + EPS * (np.abs(total) + np.abs(ref)), dtype)
    place = base.clone()
    U.balance_loss_grad(dl, x, ids, got[1], got[3], add=place, dlogits=place, **args)
    assert torch.equal(place, both) and int(host(err)[0]) == 0
