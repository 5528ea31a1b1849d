"""GPU parity of uep_gate and uep_gate_grad against the oracle (64 bits).

Ids have to be equal: softmax selects on the logits themselves, and the sigmoid cases are
drawn so that no two selection scores of a token's best are nearer than fp32 can tell (checked
on the oracle's scores).  Weights, in units eps = 2^-24 relative to the weight: one rounded
difference inside the exponential (eps times the distance d to the largest logit), expf and
sigmoid within 4 + 4 eps, a sum of E terms in any order (bounded by its longest chain,
at most E / 16 + 8 additions, times the worst term's error again), a division and a product
(4 eps).  Gradients: products and sums of at most K terms on top, relative to the sum of
magnitudes; bf16 results add half a unit, 2^-8."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle as O                                       # noqa: E402
from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, to_dev, host, say, err_word  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def draw_logits(seed, R, T, E, dtype, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = 1.5 * torch.randn(R, T, E, generator=g)
    if masked:
        x[torch.rand(R, T, E, generator=g) < masked] = -float("inf")
    return x.to(dtype)


def weight_tol(x64, E):
    finite = np.where(np.isfinite(x64), x64, 0.0)
    d = finite.max(-1, keepdims=True) - finite.min(-1, keepdims=True)
    return EPS * (2 * d + E / 16 + 40)


def run_gate(x, K, bias=None, bs=None, score=0, renorm=True, scale=1.0):
    err = err_word()
    ids, w = U.gate(x.to(DEV), K, bias=None if bias is None else to_dev(bias, torch.float32),
                    batch_size=None if bs is None else to_dev(bs), score=score, renorm=renorm,
                    scale=scale, err=err)
    return host(ids), host(w), int(host(err)[0])


def check(seed, R, T, E, K, dtype, score, renorm, scale, masked=0.0, bs=None):
    x = draw_logits(seed, R, T, E, dtype, masked)
    x64 = x.double().numpy()
    bias = (np.random.default_rng(seed).standard_normal(E) * 0.1).astype(np.float32) if score \
        else None
    ids_o, w_o = O.gate(x64, K, bias, bs, score, renorm, scale)
    if score:            # rows in which fp32 may not tell two of the best apart are made equal
        key = -np.sort(-O.gate_keys(x64, bias, score), -1)[..., :K + 1]
        with np.errstate(invalid="ignore"):
            gap = np.where(np.isfinite(key[..., 1:]), key[..., :-1] - key[..., 1:], 1.0)
        near = gap.min(-1) < 8 * EPS if gap.shape[-1] else np.zeros((R, T), bool)
        assert near.mean() < 0.05
        far = np.argwhere(~near)[0]
        x[torch.from_numpy(near)] = x[far[0], far[1]].clone()
        x64 = x.double().numpy()
        ids_o, w_o = O.gate(x64, K, bias, bs, score, renorm, scale)
    ids, w, err = run_gate(x, K, bias, bs, score, renorm, scale)
    assert err == 0
    assert np.array_equal(ids, ids_o)
    assert (np.abs(w - w_o) <= weight_tol(x64, E) * np.abs(w_o) + 1e-37).all()

    # the gradient takes the library's own weights, as a program does
    dw = np.random.default_rng(seed + 1).standard_normal((R, T, K)).astype(np.float32)
    err = err_word()
    d = U.gate_grad(to_dev(dw, torch.float32), x.to(DEV), to_dev(ids), to_dev(w, torch.float32),
                    score=score, renorm=renorm, scale=scale, err=err)
    assert int(host(err)[0]) == 0 and d.dtype == dtype
    d_o = O.gate_grad(dw, x64, ids, w, score, renorm, scale)
    on = ids >= 0
    g = np.where(on, np.abs(dw * scale), 0.0)
    s = O.gate_grad(np.zeros_like(dw), x64, ids, w, score, renorm, scale) * 0 + 1.0   # [R][T][E]
    mag = s * (g.max(-1, keepdims=True) + (np.abs(w / scale) * g).sum(-1, keepdims=True))
    if score == 0 and not renorm:      # the dense gradient scales with the expert's own score
        fin = np.where(np.isfinite(x64), x64, -np.inf)
        e = np.exp(fin - np.where(np.isfinite(fin.max(-1, keepdims=True)),
                                  fin.max(-1, keepdims=True), 0))
        mag = mag * e / np.maximum(e.sum(-1, keepdims=True), 1e-300)
    bound = weight_tol(x64, E) * mag + EPS * (K + 8) * mag + 1e-37
    if dtype == torch.bfloat16:
        bound = bound * 1.01 + 2.0 ** -8 * np.abs(d_o)
    assert (np.abs(host(d.float()) - d_o) <= bound).all()


F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("seed,R,T,E,K,dtype,score,renorm,scale,masked", [
    (0, 4, 33, 128, 8, F, 0, True, 1.0, 0.0),       # Qwen-shaped router
    (1, 2, 65, 256, 8, B, 1, True, 2.5, 0.0),       # DeepSeek-V3-shaped router
    (2, 1, 1, 128, 8, F, 0, True, 1.0, 0.0),        # one token
    (3, 1, 3, 1, 1, F, 0, False, 1.0, 0.0),         # one expert
    (4, 3, 7, 61, 4, B, 0, False, 1.0, 0.3),        # odd expert count, masked experts
    (5, 2, 19, 60, 4, F, 0, False, 0.5, 0.0),
    (6, 2, 17, 8, 8, F, 1, False, -1.5, 0.2),       # K = E, negative scale, fewer than K left
    (7, 1, 40, 200, 9, F, 1, True, 1.0, 0.1),       # K above eight
    (8, 1, 13, 513, 10, B, 0, True, 1.0, 0.0),
    (9, 2, 9, 1000, 16, F, 0, False, 1.0, 0.9),
    (10, 1, 5, 4096, 64, F, 0, True, 1.0, 0.0),     # the largest sizes
    (11, 1, 6, 3001, 33, B, 1, False, 1.0, 0.5),
    (12, 5, 31, 96, 6, B, 0, True, 1.0, 0.95),      # rows with few experts left, some with none
    (13, 7, 301, 130, 2, F, 0, True, 1.0, 0.0),
    (14, 2, 77, 24, 3, F, 0, False, 1.0, 0.05),
    (15, 1, 130, 320, 5, B, 0, False, 1.0, 0.0),
])
def test_gate_and_gradient(seed, R, T, E, K, dtype, score, renorm, scale, masked):
    say("case: gate", seed, R, T, E, K, dtype, score, renorm, scale, masked)
    check(seed, R, T, E, K, dtype, score, renorm, scale, masked)


def test_absent_tokens():
    say("case: gate batch sizes")
    check(20, 3, 50, 64, 4, F, 0, True, 1.0, bs=np.array([50, 0, 17], np.int32))
    check(21, 2, 9, 128, 8, B, 1, True, 1.0, bs=np.array([1, 8], np.int32))


@pytest.mark.parametrize("K", [1, 4, 8, 12])
def test_ties_go_to_the_lowest_id(K):
    say("case: gate ties", K)
    rng = np.random.default_rng(30 + K)
    x = torch.from_numpy(rng.integers(-2, 3, (2, 100, 128)).astype(np.float32))
    x[0, 0] = 0.0
    x[0, 1] = torch.tensor([0.0, -0.0] * 64)
    x[0, 2] = -1.5
    ids, w, err = run_gate(x, K)
    ids_o, _ = O.gate(x.double().numpy(), K)
    assert np.array_equal(ids, ids_o) and err == 0
    assert ids[0, 0].tolist() == list(range(K)) == ids[0, 1].tolist()


@pytest.mark.parametrize("dtype", [F, B])
def test_special_logits(dtype):
    """-infinity masks, NaN and +infinity mask and are flagged, the type's lowest value is an
    ordinary logit (selected last), and so are values whose exponentials underflow."""
    say("case: gate special logits", dtype)
    inf, low = float("inf"), torch.finfo(dtype).min
    E, K = 16, 4
    x = torch.full((1, 8, E), -inf)
    x[0, 1, 3], x[0, 1, 9] = low, 1.0                   # two left, one of them the lowest value
    x[0, 2] = low                                        # all the lowest value: uniform
    x[0, 3, :5] = torch.tensor([5.0, -200.0, -201.0, 4.0, -202.0])
    x[0, 4] = torch.arange(E, dtype=torch.float32)
    x = x.to(dtype)
    for score in (0, 1):
        for renorm in (True, False):
            ids, w, err = run_gate(x, K, score=score, renorm=renorm)
            ids_o, w_o = O.gate(x.double().numpy(), K, score=score, renorm=renorm)
            assert err == 0
            if score == 0:
                assert np.array_equal(ids, ids_o)
                assert (np.abs(w - w_o) <= 1e-6 * w_o + 1e-37).all()
            assert (ids[0, 0] == -1).all() and (w[0, 0] == 0).all()
            assert np.isfinite(w).all()
            dw = torch.ones(1, 8, K, device=DEV)
            d = host(U.gate_grad(dw, x.to(DEV), to_dev(ids), to_dev(w, torch.float32),
                                 score=score, renorm=renorm).float())
            assert np.isfinite(d).all() and (d[0, 0] == 0).all()
            assert (d[0][~np.isfinite(x[0].float().numpy())] == 0).all()
    y = x.clone()
    y[0, 4, 15], y[0, 4, 14], y[0, 5, 2] = float("nan"), inf, inf
    ids, w, err = run_gate(y, K)
    assert err == U.ERR_LOGIT
    assert ids[0, 4].tolist() == [13, 12, 11, 10] and (ids[0, 5] == -1).all()
    assert np.isfinite(w).all()


@pytest.mark.parametrize("E,K", [(16, 1), (16, 4), (40, 20)])
def test_renormalised_weights_of_tiny_scores(E, K):
    """Sigmoid scores near the smallest fp32 number still share out the scale."""
    say("case: gate tiny scores", E, K)
    x = torch.full((1, 3, E), -87.0)
    x[0, 1] = -86.5
    x[0, 2, ::2] = -86.9
    _, w, err = run_gate(x, K, score=1, renorm=True, scale=50.0)
    assert err == 0 and np.abs(w.sum(-1) - 50.0).max() < 50.0 * (K + 40) * EPS


def test_bias_may_mask_experts():
    say("case: gate bias masks")
    x = torch.arange(12, dtype=torch.float32).view(1, 1, 12) / 4
    bias = np.zeros(12, np.float32)
    bias[[11, 10]] = -np.inf
    ids, _, err = run_gate(x, 3, bias=bias, score=1)
    assert ids[0, 0].tolist() == [9, 8, 7] and err == 0
    bias[9] = np.nan
    ids, _, err = run_gate(x, 3, bias=bias, score=1)
    assert ids[0, 0].tolist() == [8, 7, 6] and err == U.ERR_LOGIT


def test_gradient_skips_bad_ids_and_writes_every_element():
    say("case: gate_grad ids out of range")
    R, T, E, K = 1, 3, 40, 3
    x = draw_logits(40, R, T, E, F)
    ids, w, _ = run_gate(x, K)
    bad = ids.copy()
    bad[0, 1, 1], bad[0, 2, 0] = E, -7
    for renorm, score in ((True, 0), (False, 0), (True, 1), (False, 1)):
        err = err_word()
        d = torch.full((R, T, E), float("nan"), device=DEV)
        U.gate_grad(torch.ones(R, T, K, device=DEV), x.to(DEV), to_dev(bad),
                    to_dev(w, torch.float32), score=score, renorm=renorm, dlogits=d, err=err)
        assert int(host(err)[0]) == U.ERR_ID_RANGE
        assert np.isfinite(host(d)).all()


def test_unaligned_views_and_other_streams():
    """A logits view that starts at an odd element, and calls on another stream."""
    say("case: gate unaligned")
    for dtype in (F, B):
        flat = draw_logits(50, 1, 1, 1 + 6 * 128, dtype).view(-1).to(DEV)
        x = flat[1:].view(1, 6, 128)
        ids0, w0 = U.gate(x.clone(), 8)
        ids1, w1 = U.gate(x, 8)
        assert torch.equal(ids0, ids1) and torch.equal(w0, w1)
        out = torch.zeros(1 + 6 * 128, dtype=dtype, device=DEV)
        dw = torch.randn(1, 6, 8, device=DEV)
        d0 = U.gate_grad(dw, x.clone(), ids0, w0, renorm=False)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        U.gate_grad(dw, x, ids0, w0, renorm=False, dlogits=out[1:], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out[1:].view(1, 6, 128), d0) and float(out[0]) == 0


def test_captured_graph_replays():
    say("case: gate in a graph")
    x = draw_logits(60, 2, 300, 128, F).to(DEV)
    ids = torch.empty(2, 300, 8, dtype=torch.int32, device=DEV)
    w = torch.empty(2, 300, 8, device=DEV)
    dw = torch.randn(2, 300, 8, device=DEV)
    dl = torch.empty_like(x)
    U.gate(x, 8, topk_ids=ids, gate_w=w)
    U.gate_grad(dw, x, ids, w, dlogits=dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        U.gate(x, 8, topk_ids=ids, gate_w=w)
        U.gate_grad(dw, x, ids, w, dlogits=dl)
    for seed in (61, 62, 63):
        x.copy_(draw_logits(seed, 2, 300, 128, F).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        i2, w2 = U.gate(x, 8)
        assert torch.equal(ids, i2) and torch.equal(w, w2)
        assert torch.equal(dl, U.gate_grad(dw, x, i2, w2))


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_keeps_its_digits(dtype, renorm):
    """Scores near 1, where the difference 1 - s loses its digits (at a logit of 12 it is 1 % off,
    from 17 on it is 0).  The bound is relative to the gradient: 1 - s by its exponential
    |l| + 2 <= 82 units of 2^-24, its sum and reciprocal 3, the weight without its scale 1, the
    scaled dw 1, the dot product K + 1, the products 3; the four weights are alike, so that no
    difference of theirs cancels by more than two bits (4 + 4).  104 in all."""
    say("case: gate_grad, scores near one", dtype, renorm)
    E, K = 64, 4
    x = torch.full((1, 12, E), -20.0)
    for t, top in enumerate((3.0, 8.0, 10.0, 12.0, 14.0, 16.0, 17.0, 18.0, 22.0, 30.0, 50.0, 80.0)):
        x[0, t, torch.tensor([9, 33, 5, 60])] = torch.tensor([top, top - 0.5, top - 1.0, top - 2.0])
    x = x.to(dtype)
    ids, w, err = run_gate(x, K, score=1, renorm=renorm, scale=2.5)
    assert err == 0 and sorted(ids[0, 0].tolist()) == [5, 9, 33, 60]
    ids = np.broadcast_to(np.array([9, 33, 5, 60], np.int32), ids.shape)
    s = 1.0 / (1.0 + np.exp(-np.take_along_axis(x.double().numpy(), ids, -1)))
    w = (2.5 * (s / s.sum(-1, keepdims=True) if renorm else s)).astype(np.float32)
    for k in range(K):
        dw = np.zeros((1, 12, K), np.float32)
        dw[..., k] = 1.25
        d = host(U.gate_grad(to_dev(dw, torch.float32), x.to(DEV), to_dev(ids),
                             to_dev(w, torch.float32), score=1, renorm=renorm, scale=2.5).float())
        want = O.gate_grad(dw, x.double().numpy(), ids, w, 1, renorm, 2.5)
        tol = EPS * 104 + (2.0 ** -8 if dtype == B else 0.0)
        assert (np.abs(d - want) <= tol * np.abs(want)).all()
        assert (d != 0).sum() == 12 * (K if renorm else 1)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("R,T,E,K", [
    (1, 9, 64, 1), (2, 300, 40, 4), (1, 50, 300, 8), (1, 21, 40, 20), (1, 17, 1100, 8),
    (3, 3001, 128, 8), (2, 4500, 256, 16),                       # more than 8192 tokens
])
def test_sigmoid_without_a_bias_orders_by_the_logits(dtype, R, T, E, K):
    """Without a bias the scores' order is the logits' order, also where scores that differ are
    the same fp32 number: 1 above a logit of 17, 0 below -88."""
    say("case: gate, sigmoid without a bias", dtype, R, T, E, K)
    g = torch.Generator().manual_seed(70 + E)
    x = 40.0 * torch.randn(R, T, E, generator=g)
    x[0, 0, :2] = torch.tensor([17.5, 30.0])
    x[0, 0, 2:] = 1.0
    x[0, 1] = -90.0 - torch.arange(E)
    x[0, 2] = 20.0 + torch.arange(E)
    x[0, 3, ::2] = -float("inf")
    x[0, 4, :] = torch.tensor([0.0, -0.0] * (E // 2))
    x = x.to(dtype)
    x64 = x.double().numpy()
    for renorm in (True, False):
        ids, w, err = run_gate(x, K, score=1, renorm=renorm, scale=1.5)
        ids_o, w_o = O.gate(x64, K, score=1, renorm=renorm, scale=1.5)
        assert err == 0
        assert np.array_equal(ids, ids_o)
        top = np.take_along_axis(x64, np.maximum(ids_o, 0), -1).max(-1)
        near = top > -80                            # scores below 2^-126 count as 0
        tol = EPS * (2 * 88 + 40) * np.abs(w_o) + 1e-37
        assert (np.abs(w - w_o) <= tol)[near].all()
        assert np.isfinite(w).all()


def test_the_most_tokens():
    """2^26 - 1 tokens, the documented limit, by the kernel that takes a wave for each."""
    n = 2 ** 26 - 1
    say("case: gate, 2^26 - 1 tokens")
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of device memory")
    g = torch.Generator(device=DEV).manual_seed(90)
    x = torch.randn(1, n, 2, generator=g, device=DEV)
    bs = to_dev(np.array([n - 3]))
    ids, w = U.gate(x, 1, batch_size=bs)
    want = (x[..., 1:] > x[..., :1]).to(torch.int32)
    assert torch.equal(ids[:, :n - 3], want[:, :n - 3])
    assert bool((w[:, :n - 3] == 1).all())
    assert bool((ids[:, n - 3:] == -1).all()) and bool((w[:, n - 3:] == 0).all())
    del x, ids, w, want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E,K", [(40, 4), (40, 20), (1100, 3)])
def test_a_bias_is_checked_behind_a_masked_logit(E, K):
    """A bias that is not a number is flagged whatever its expert's logit, at every size."""
    say("case: gate, bias behind a masked logit", E, K)
    x = draw_logits(80, 1, 3, E, F)
    x[..., 7] = -float("inf")
    for value, want in ((float("nan"), U.ERR_LOGIT), (float("inf"), U.ERR_LOGIT),
                        (-float("inf"), 0), (0.5, 0)):
        bias = np.zeros(E, np.float32)
        bias[7] = value
        ids, w, err = run_gate(x, K, bias=bias, score=1)
        assert err == want, value
        assert (ids != 7).all() and (ids >= 0).all() and np.isfinite(w).all()


def busy():
    """Work on the current stream that takes some 20 ms, and no answer from the device."""
    x = torch.empty(1 << 28, device=DEV)
    for _ in range(100):
        x.fill_(1.0)


def test_outputs_for_another_stream():
    """Outputs that a call allocates for `stream` are not touched by what the current stream
    still has to do with the same memory."""
    say("case: gate, outputs for another stream")
    x = draw_logits(95, 1, 4000, 64, F).to(DEV)
    ids0, w0 = U.gate(x, 8)
    d0 = U.gate_grad(w0, x, ids0, w0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, want in ((lambda: U.gate(x, 8, stream=side), (ids0, w0)),
                       (lambda: (U.gate_grad(w0, x, ids0, w0, stream=side),), (d0,))):
        old = [torch.empty_like(t) for t in want]
        busy()
        for t in old:
            t.fill_(7)
        t = old = None                                           # freed, the fills still queued
        got = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("R,T,E,K,dtype,score,renorm,masked", [
    (1, 70001, 27, 8, F, 0, True, 0.1),         # a wave's second group of 8 tokens
    (1, 70001, 27, 8, B, 0, False, 0.0),        # the same, dense
    (1, 70001, 30, 7, F, 1, False, 0.0),
    (1, 70001, 30, 7, B, 1, True, 0.3),
    (3, 11003, 61, 9, F, 0, False, 0.2),        # second and third groups of 4 tokens
    (3, 11003, 61, 9, B, 1, True, 0.0),
    (1, 20001, 70, 33, F, 0, True, 0.0),        # a token a wave, up to three turns
    (1, 20001, 70, 33, B, 0, False, 0.1),
    (1, 8200, 1111, 40, F, 0, False, 0.0),      # rows over more than one window
    (1, 8200, 1111, 40, B, 1, False, 0.0),
])
def test_gradient_of_many_tokens(R, T, E, K, dtype, score, renorm, masked):
    """More groups of tokens than waves, which take the next with the window of the last."""
    say("case: gate_grad, many tokens", R, T, E, K, dtype, score, renorm, masked)
    check(200 + E + K, R, T, E, K, dtype, score, renorm, 1.0, masked)


# The sorting kernel's forms above 8192 tokens: 4 lanes of 32 or 64 experts and 8 of 64, with
# lists of 4, 8 and 16 (above 512 experts 16 lanes of 64 at any number of tokens); 61, 324 and
# 702 end inside a 16-byte vector of at least one type.
@pytest.mark.parametrize("E", [61, 128, 200, 256, 324, 512, 702])
@pytest.mark.parametrize("K", [3, 8, 16])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("score", [0, 1])
def test_gate_of_many_tokens(E, K, dtype, score):
    say("case: gate, many tokens", E, K, dtype, score)
    seed, T = E * 64 + K * 4 + score, 2801 if E <= 512 else 301
    check(seed, 3, T, E, K, dtype, score, True, 2.5, 0.0)
    check(seed + 1, 3, T, E, K, dtype, score, False, 1.0, 0.97 if E > 200 else 0.6,
          bs=np.array([T, 0, T - 77], np.int32))


@pytest.mark.parametrize("E", [60, 128, 256, 384, 512, 1024])
@pytest.mark.parametrize("K", [1, 8, 13])
@pytest.mark.parametrize("dtype", [F, B])
def test_ties_and_special_logits_of_many_tokens(E, K, dtype):
    """Whole numbers tie often; ids are those of the oracle to the last, with -0, -infinity, the
    type's lowest value, +infinity and NaN among them, by the logits and with a bias that only
    masks (scores of whole numbers below 9 are far apart)."""
    say("case: gate, ties of many tokens", E, K, dtype)
    rng = np.random.default_rng(E + K)
    T = 4600 if E <= 512 else 600
    x = torch.from_numpy(rng.integers(-8, 9, (2, T, E)).astype(np.float32))
    x[0, 0], x[0, 1], x[0, 2] = 0.0, -float("inf"), torch.finfo(dtype).min
    x[0, 3] = torch.tensor([0.0, -0.0] * (E // 2))
    x[0, 4, 5:] = -float("inf")
    x[1, :, 3] = -float("inf")
    x = x.to(dtype)
    bias = np.where(np.arange(E) % 5 == 1, -np.inf, 0.0).astype(np.float32)
    for score, b in ((0, None), (1, None), (1, bias)):
        ids, w, err = run_gate(x, K, bias=b, score=score)
        y = x.double()
        if b is not None:                # the lowest value's score is 0, and 0 ties with 0
            y = y.clamp(min=-100.0).masked_fill(x == -float("inf"), -float("inf"))
        assert err == 0 and np.array_equal(ids, O.gate(y.numpy(), K, b, score=score)[0])
        assert np.isfinite(w).all() and ((ids >= 0) | (w == 0)).all()
    bad = x.clone()
    bad[1, 77, 1], bad[1, T - 1, E - 1] = float("nan"), float("inf")
    ids, w, err = run_gate(bad, K)
    assert err == U.ERR_LOGIT and np.array_equal(ids, O.gate(bad.double().numpy(), K)[0])
    assert np.isfinite(w).all()


@pytest.mark.parametrize("E,K", [(40, 17), (256, 24), (300, 20), (1000, 33), (1024, 64), (1025, 1),
                                 (7, 5), (3, 2)])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("score", [0, 1])
def test_gate_of_many_slots_or_few_experts(E, K, dtype, score):
    say("case: gate, many slots", E, K, dtype, score)
    for renorm in (True, False):
        check(E + K, 2, 90, E, K, dtype, score, renorm, 1.5, 0.3, bs=np.array([90, 31], np.int32))


def test_calls_follow_the_current_stream(monkeypatch):
    """Without `stream` a call goes to the current one, by either way of asking torch for it."""
    say("case: gate, the current stream")
    assert U._RAW_STREAM is not None
    x = draw_logits(97, 1, 3000, 128, F).to(DEV)
    want = U.gate(x, 8)
    side = torch.cuda.Stream()
    for raw in (U._RAW_STREAM, None):
        monkeypatch.setattr(U, "_RAW_STREAM", raw)
        assert (U._s(None).value or 0) == torch.cuda.current_stream().cuda_stream
        late = torch.zeros_like(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            assert U._s(None).value == side.cuda_stream
            busy()
            late.copy_(x)                                        # queued on `side` before the call
            got = U.gate(late, 8)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F, B])
def test_sigmoid_gradient_where_its_two_forms_meet(dtype):
    """Logits from -8 to 12 without renormalisation, with the library's own weights: 1 - s by the
    weight, whose 6 units of 2^-24 are at most 6 * 64 of it (6 * 256 for bf16), or by the logit (17
    units up to 12), and 18 for the other factors, relative to the gradient."""
    say("case: gate_grad, sigmoid from -8 to 12", dtype)
    E, K, T = 16, 4, 2000
    x = torch.linspace(-8, 12, T).view(1, T, 1) - 0.01 * torch.arange(E).view(1, 1, E)
    x = x.to(dtype)
    ids, w, err = run_gate(x, K, score=1, renorm=False, scale=2.5)
    dw = np.random.default_rng(99).uniform(0.5, 1.5, (1, T, K)).astype(np.float32)
    d = host(U.gate_grad(to_dev(dw, torch.float32), x.to(DEV), to_dev(ids),
                         to_dev(w, torch.float32), score=1, renorm=False, scale=2.5).float())
    x64 = x.double().numpy()
    s = 1 / (1 + np.exp(-np.take_along_axis(x64, ids, -1)))
    want = O.gate_grad(dw, x64, ids, 2.5 * s, 1, False, 2.5)
    tol = EPS * (6 * 64 + 18) if dtype == F else EPS * (6 * 256 + 18) + 2.0 ** -8
    assert err == 0 and (np.abs(d - want) <= tol * np.abs(want)).all()
    assert ((d != 0).sum(-1) == K).all()
