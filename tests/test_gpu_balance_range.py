"""The balance loss' gradient at the ends of its range, against the oracle in 64 bits.

The gradient is f p_e (c_e - sum_j p_j c_j) [(1 - s_e)] with f = dloss E / (K n^2).  A kernel may
subtract any c_0 from the counts first; with the integer next to sum_j p_j c_j, and eps = 2^-24, a
score within rel (4 spread + 160 eps, spread the largest distance or logit) and at most 75
additions, the sum is within (rel + 75 eps) sum_j p_j |c_j - c_0|, and the difference's, the four
products' and f's roundings and 1 - s (another score) are within (2 rel + 16 eps) of the result."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle as O                                       # noqa: E402
from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, to_dev, host, say, err_word   # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def spread(x, score):
    """Largest finite logit, or distance to a row's largest."""
    f = np.where(np.isfinite(x), x, np.nan).reshape(-1, x.shape[-1])
    return float(np.nanmax(np.abs(f)) if score else np.nanmax(np.nanmax(f, -1) - np.nanmin(f, -1)))


def oracle_and_room(dloss, x, ids, counts, tokens, G, off, score):
    """The gradient, and how far a call may be from it before it is stored."""
    E, K = x.shape[-1], ids.shape[-1]
    ref = O.balance_loss_grad(dloss, x, ids, counts, tokens, G, off, score)
    p, _ = O.balance_shares(x, score)
    rel = (4 * spread(x, score) + 160) * EPS
    room = (2 * rel + 16 * EPS) * np.abs(ref).reshape(p.shape)
    for g, (a, b) in enumerate(O.balance.spans(len(p), G, off)):
        n = float(tokens[g])
        if n <= 0 or a == b:
            continue
        c = np.asarray(counts[g], dtype=np.float64)
        c0 = np.rint(p[a:b] @ c)[:, None]
        sums = (p[a:b] * np.abs(c - c0)).sum(-1, keepdims=True)
        room[a:b] += abs(float(dloss[g])) * E / (K * n * n) * p[a:b] * (rel + 75 * EPS) * sums
    return ref, room.reshape(ref.shape)


def check(d, ref, room, dtype=torch.float32):
    got, half = d.double().cpu().numpy(), torch.finfo(dtype).eps / 2
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= room + half * (np.abs(ref) + room) + 2.0 ** -133).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("left", [(-87.0,), (-86.0, -87.0), (-80.0, -86.5, -84.0), (-40.0, 3.0)])
@pytest.mark.parametrize("dloss", [1.0, 1e20])
def test_scores_at_the_bottom_of_their_range(left, dloss, dtype):
    """Sigmoid scores of which all that are left are near 2^-126: their shares are numbers like any
    others, and so is the gradient (0 where one expert is left)."""
    say("case: tiny scores", left, dloss, dtype)
    E = 4096
    x = torch.full((1, 3, E), -float("inf"), device=DEV)
    x[0, :, 100:100 + len(left)] = torch.tensor(left, device=DEV)
    x = x.to(dtype)
    ids = torch.full((1, 3, 1), 100, dtype=torch.int32, device=DEV)
    err = err_word()
    _, counts, _, tokens = U.balance_loss(x, ids, 3, score=U.GATE_SIGMOID, err=err)
    each = [dloss, -dloss, dloss]
    d = U.balance_loss_grad(to_dev(np.array(each), torch.float32), x, ids, counts, tokens,
                            score=U.GATE_SIGMOID, err=err)
    ref, room = oracle_and_room(np.float32(each), x.double().cpu().numpy(), host(ids), host(counts),
                                host(tokens), 3, None, 1)
    check(d, ref, room, dtype)
    assert int(host(err)[0]) == 0 and (ref != 0).any() == (len(left) > 1)


@pytest.mark.parametrize("score", [U.GATE_SOFTMAX, U.GATE_SIGMOID])
@pytest.mark.parametrize("E,K", [(2, 1), (16, 8), (60, 16), (1500, 40)])
@pytest.mark.parametrize("near", [1, 3000, 1 << 20])
def test_counts_past_24_bits(E, K, near, score):
    """Counts of a whole group, far past 2^24 and near each other: what tells them apart are their
    differences, and those are exact."""
    say("case: large counts", E, K, near, score)
    rng = np.random.default_rng(E + near)
    n = min(1 << 26, (1 << 30) // K)
    near = min(near, K * n // E - 1)
    counts = (K * n // E + rng.integers(-near, near + 1, (2, E))).astype(np.int32)
    x = to_dev(rng.normal(size=(1, 60, E)) * 2, torch.float32)
    ids = to_dev(rng.integers(0, E, (1, 60, K)))
    tokens, dloss = np.array([n, n - 5], np.int32), np.float32([1e9, -3e8])
    d = U.balance_loss_grad(to_dev(dloss, torch.float32), x, ids, to_dev(counts), to_dev(tokens),
                            score=score)
    ref, room = oracle_and_room(dloss, host(x).astype(np.float64), host(ids), counts, tokens, 2, None,
                                score)
    check(d, ref, room)


@pytest.mark.parametrize("score", [U.GATE_SOFTMAX, U.GATE_SIGMOID])
def test_two_busy_experts_of_many(score):
    """Two experts with nearly all ids and nearly all of p, the others with none: their counts
    differ by one, and that is what their gradients are made of."""
    E = 64
    x = torch.full((1, 8, E), -30.0, device=DEV)
    x[..., 7] = x[..., 50] = 0.5
    ids = torch.tensor([7, 50], dtype=torch.int32, device=DEV).expand(1, 8, 2).contiguous()
    counts = np.zeros((1, E), np.int32)
    counts[0, 7], counts[0, 50] = (1 << 30) - 1, 1 << 30
    tokens = np.array([1 << 30], np.int32)
    d = U.balance_loss_grad(torch.full((1,), 1e18, device=DEV), x, ids, to_dev(counts),
                            to_dev(tokens), score=score)
    ref, room = oracle_and_room(np.float32([1e18]), host(x).astype(np.float64), host(ids), counts,
                                tokens, 1, None, score)
    check(d, ref, room)
