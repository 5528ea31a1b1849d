"""GPU parity of the AdamW step against the oracle: fp32 states, 8-bit codes and tops bit
for bit; parameters to 2^-24 (4 |p| + 24 |change|) (p's product with the decay, the decay's
own two roundings and the last subtraction act on |p|; root, quotients and factors, each good
to two units, on the change); bf16 parameters are one of the bit patterns that the random cut
of a value within that bound gives."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from oracle import adamw as A                            # noqa: E402
from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, host, say, err_word   # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
F, B = torch.float32, torch.bfloat16
SIZES = [1, 3, 256, 257, 4096, 5000, 12289, 0, 70000, 2]


def place(x, dtype, shift):
    """x on the device as `dtype`, `shift` elements into its allocation."""
    x = torch.as_tensor(x).to(dtype)
    t = torch.zeros(x.numel() + shift, dtype=dtype, device=DEV)[shift:]
    t.copy_(x)
    return t


def draw(rng, n, param, grad, eight, shift):
    spread = np.exp(2 * rng.standard_normal(n))
    p = place(0.05 * rng.standard_normal(n), param, shift)
    g = place(1e-3 * spread * rng.standard_normal(n), grad, shift)
    m = (3e-4 * spread * rng.standard_normal(n)).astype(np.float32)
    v = ((1e-3 * spread) ** 2 * rng.random(n)).astype(np.float32)
    if n > 8:
        g[2], m[3], v[3], g[3] = 0.0, 0.0, 0.0, 0.0        # an element that has not moved yet
    tops = None
    if eight:
        z = rng.integers(0, 1 << 16, n, dtype=np.uint32)
        m, v, tops = A.encode(m, v, z, z)
        tops = place(tops, torch.int32, 0)
    st = torch.uint8 if eight else F
    return p, g, place(m, st, shift), place(v, st, shift), tops


def bf16_bits(t):
    return host(t.view(torch.int16)).view(np.uint16)


def bf16_order(bits):
    """bf16 bit patterns as integers in the order of their values (both zeros 0)."""
    b = bits.astype(np.int64)
    return np.where(b & 0x8000, -(b & 0x7FFF), b)


def check_step(params, grads, ms, vs, tops, copies, step, lr, factor, wd, ls, betas, eps, seed,
               err_want=0):
    eight = tops is not None
    before = [[host(t).copy() if t.dtype != B else host(t.float()).copy() for t in x]
              for x in (params, grads, ms, vs)]
    tops0 = [host(t).copy() for t in tops] if eight else None
    err = err_word()
    plan = U.adamw_prepare(params, grads, ms, vs, copies=copies, tops=tops, weight_decay=wd,
                           lr_scale=ls)
    sched = torch.tensor([lr, factor], device=DEV)
    U.adamw(plan, torch.tensor([step], dtype=torch.int32, device=DEV), sched, beta1=betas[0],
            beta2=betas[1], eps=eps, seed=seed, err=err)
    assert int(host(err)[0]) == err_want
    for i in range(len(params)):
        n = params[i].numel()
        if n == 0:
            continue
        p0, g, m0, v0 = (x[i] for x in before)
        if eight:
            m0, v0 = A.decode(m0, v0, tops0[i])
        m, v, _ = A.moments(g, m0, v0, factor, *betas)
        dp, dm, dv = A.dithers(seed, step, i, n)
        if eight:
            cm, cv, t = A.encode(m, v, dm, dv)
            assert np.array_equal(host(ms[i]), cm) and np.array_equal(host(vs[i]), cv), i
            assert np.array_equal(host(tops[i]), t), i
            dm8, dv8 = U.adamw_decode(ms[i].clone(), vs[i].clone(), tops[i])
            hm, hv = A.decode(cm, cv, t)
            assert np.array_equal(host(dm8), hm) and np.array_equal(host(dv8), hv)
            dm8, dv8 = U.adamw_decode(ms[i].clone(), vs[i].clone(), tops[i], dtype=B)
            assert np.array_equal(host(dm8.float()), hm) and np.array_equal(host(dv8.float()), hv)
        else:
            assert np.array_equal(host(ms[i]), m) and np.array_equal(host(vs[i]), v), i
        lr32 = float(np.float32(lr) * np.float32(ls[i]))
        w, change = A.update(p0, m, v, step, lr32, wd[i], *betas, eps)
        tol = EPS * (4 * np.abs(p0) + 24 * change) + 1e-37
        if params[i].dtype == F:
            got = host(params[i])
            assert (np.abs(got - w) <= tol).all(), i
            if copies is not None:
                assert torch.equal(copies[i], params[i].to(B)), i
        else:
            got = bf16_bits(params[i])
            lo, hi = A.cut_bf16((w - tol).astype(np.float32), dp), A.cut_bf16(
                (w + tol).astype(np.float32), dp)
            lo, got, hi = (bf16_order(x) for x in (lo, got, hi))
            assert ((lo <= got) & (got <= hi)).all(), i
            assert (hi - lo <= 1).mean() > 0.999           # nearly always one or two patterns


@pytest.mark.parametrize("param", [F, B])
@pytest.mark.parametrize("grad", [F, B])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_step(param, grad, eight, shift):
    say("case: adamw", param, grad, eight, shift)
    rng = np.random.default_rng(100)
    sets = [draw(rng, n, param, grad, eight, shift) for n in SIZES]
    params, grads, ms, vs, tops = (list(x) for x in zip(*sets))
    copies = [torch.zeros(n + shift, dtype=B, device=DEV)[shift:] for n in SIZES] \
        if param == F else None
    k = len(SIZES)
    for step in (1, 2, 1000):
        check_step(params, grads, ms, vs, tops if eight else None, copies, step, 1e-3, 0.5,
                   [0.1 * (i % 2) for i in range(k)], [1.0 + i % 3 for i in range(k)],
                   (0.9, 0.999), 1e-8, 77 + step)


def test_other_betas_and_many_tensors():
    say("case: adamw, betas of 0, many tensors")
    rng = np.random.default_rng(101)
    sets = [draw(rng, int(n), F, F, False, 0) for n in rng.integers(1, 700, 300)]
    params, grads, ms, vs, _ = (list(x) for x in zip(*sets))
    check_step(params, grads, ms, vs, None, None, 3, 1e-2, 1.0, [0.0] * 300, [1.0] * 300,
               (0.0, 0.5), 1e-5, 0)


@pytest.mark.parametrize("eight", [False, True])
def test_gradients_that_are_not_finite(eight):
    say("case: adamw, gradients not finite", eight)
    rng = np.random.default_rng(102)
    p, g, m, v, tops = draw(rng, 3000, F, F, eight, 0)
    g[5], g[700], g[2999] = float("nan"), float("inf"), -float("inf")
    check_step([p], [g], [m], [v], [tops] if eight else None, None, 4, 1e-3, 1.0, [0.1], [1.0],
               (0.9, 0.999), 1e-8, 5, err_want=U.ERR_GRAD)
    assert torch.isfinite(p).all()


def test_huge_and_tiny_gradients_in_8_bits():
    """Squares that overflow keep the largest level, squares that underflow are zero, and no
    parameter stops being a number."""
    say("case: adamw 8 bits, extreme gradients")
    g = np.zeros(1024, dtype=np.float32)
    g[:256] = 1e30
    g[256:512] = 1e-30
    g[512:768:2] = 1e18
    g[512] = 1.0
    z = torch.zeros(1024, dtype=torch.uint8, device=DEV)
    p = torch.ones(1024, device=DEV)
    m, v, tops = z.clone(), z.clone(), torch.zeros(4, dtype=torch.int32, device=DEV)
    for step in (1, 2):
        check_step([p], [place(g, F, 0)], [m], [v], [tops], None, step, 1e-3, 1.0, [0.0], [1.0],
                   (0.9, 0.999), 1e-8, 9)
    assert torch.isfinite(p).all()


def test_second_moments_below_the_normal_range():
    """Squares around 2^-126 with an eps of 1e-30: the root of a subnormal number counts."""
    say("case: adamw, subnormal second moments")
    rng = np.random.default_rng(105)
    n = 5000
    g = (10.0 ** rng.uniform(-22, -18, n) * rng.choice([-1, 1], n)).astype(np.float32)
    z = torch.zeros(n, device=DEV)
    check_step([torch.ones(n, device=DEV)], [place(g, F, 0)], [z], [z.clone()], None, None, 1,
               1e-3, 1.0, [0.0], [1.0], (0.9, 0.999), 1e-30, 0)


def test_overlapping_tensors_are_refused():
    """Tensors that one step would write twice, and gradients inside what it writes."""
    say("case: adamw overlaps")
    x = torch.zeros(4000, device=DEV)
    p, m, v, g = x[:1000], x[1000:2000], x[2000:3000], x[3000:]
    U.adamw_prepare([p], [g], [m], [v])
    U.adamw_prepare([p[:500], p[500:]], [g[:500], g[:500]], [m[:500], m[500:]], [v[:500], v[500:]])
    for args, match in ((([p], [g], [x[999:1999]], [v]), "overlap"),
                        (([p, p], [g, g], [m, m.clone()], [v, v.clone()]), "overlap"),
                        (([p], [x[2001:3001]], [m], [v]), "grads.0. overlaps v.0."),
                        (([p], [x[500:1500]], [m], [v]), "grads.0. overlaps"),
                        (([p], [p], [m], [v]), "grads.0. overlaps params.0.")):
        with pytest.raises(TypeError, match=match):
            U.adamw_prepare(*args)


def test_plan_errors_leave_everything_alone():
    say("case: adamw plan errors")
    p, g, m, v = (torch.ones(500, device=DEV) for _ in range(4))
    plan = U.adamw_prepare([p], [g], [m], [v])
    sched = torch.tensor([0.1, 1.0], device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    for what in ("step", "types", "buffer"):
        err = err_word()
        if what == "step":
            U.adamw(plan, torch.zeros(1, dtype=torch.int32, device=DEV), sched, err=err)
        else:
            import dataclasses
            other = dataclasses.replace(plan, grad_dtype=U.BF16) if what == "types" else \
                dataclasses.replace(plan, buf=torch.zeros_like(plan.buf))
            U.adamw(other, one, sched, err=err)
        assert int(host(err)[0]) == U.ERR_PLAN
        assert all(bool((t == 1).all()) for t in (p, m, v))


def test_second_moments_decay_in_8_bits():
    """1000 steps without a gradient: v falls to beta2^1000 = 0.368 of itself, which rounding
    to nearest would never do (one step is 0.1 %, half a level 3 %).  Stochastic rounding is
    exact in the mean; over 65536 elements the mean's standard error is below
    0.02 (a level's variance a step, summed, over sqrt(65536)): 0.1 is allowed."""
    say("case: adamw 8 bits, decay")
    n = 65536
    rng = np.random.default_rng(103)
    v0 = np.exp(rng.uniform(-3, 0, n)).astype(np.float32)
    z = np.full(n, 1 << 15, dtype=np.uint32)
    cm, cv, tops = A.encode(np.zeros(n, np.float32), v0, z, z)
    m, v, t = place(cm, torch.uint8, 0), place(cv, torch.uint8, 0), place(tops, torch.int32, 0)
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    plan = U.adamw_prepare([p], [g], [m], [v], tops=[t])
    sched = torch.tensor([1e-3, 1.0], device=DEV)
    step = torch.zeros(1, dtype=torch.int32, device=DEV)
    start = float(U.adamw_decode(m, v, t)[1].double().mean())
    for _ in range(1000):
        step += 1
        U.adamw(plan, step, sched, seed=3)
    end = float(U.adamw_decode(m, v, t)[1].double().mean())
    assert abs(end / start / 0.999 ** 1000 - 1) < 0.1


def test_captured_graph_takes_new_steps_and_rates():
    say("case: adamw in a graph")
    g0 = torch.Generator(device=DEV).manual_seed(4)
    a = [torch.randn(9000, generator=g0, device=DEV) for _ in range(2)] + \
        [torch.zeros(9000, device=DEV) for _ in range(2)]
    b = [x.clone() for x in a]
    pa, pb = U.adamw_prepare(*[[x] for x in a]), U.adamw_prepare(*[[x] for x in b])
    step = torch.zeros(1, dtype=torch.int32, device=DEV)
    sched = torch.tensor([0.0, 1.0], device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        U.adamw(pa, step, sched)
    for t in range(1, 5):
        step.fill_(t)
        sched[0] = 1e-3 * t
        graph.replay()
        torch.cuda.synchronize()
        U.adamw(pb, step, sched)
        assert all(torch.equal(x, y) for x, y in zip(a, b)), t


def test_offsets_past_32_bits():
    """bf16 parameters and gradients with 8-bit states, 2^31 + 300 elements: the tail is
    stepped like the same elements of the oracle."""
    say("case: adamw, more than 2^31 elements")
    n = 2 ** 31 + 300
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    rng = np.random.default_rng(104)
    p, g = (torch.zeros(n, dtype=B, device=DEV) for _ in range(2))
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    tops = torch.zeros(-(-n // 256), dtype=torch.int32, device=DEV)
    k = 300 + 256 * 5                                            # whole blocks up to the end
    g[n - k:] = torch.from_numpy(rng.standard_normal(k)).to(B).to(DEV)
    g[:512] = 1.0
    plan = U.adamw_prepare([p], [g], [m], [v], tops=[tops])
    U.adamw(plan, torch.ones(1, dtype=torch.int32, device=DEV),
            torch.tensor([1e-3, 1.0], device=DEV), seed=1)
    tail = host(g[n - k:].float())
    mo, vo, _ = A.moments(tail, np.zeros(k, np.float32), np.zeros(k, np.float32), 1.0)
    i = np.arange(n - k, n, dtype=np.uint64)
    # the oracle's random words of these groups alone
    key = A._mix(A._mix(np.uint64((0x9E3779B9 + 1) & 0xFFFFFFFF)) ^ np.uint64(1))
    w = [A._mix((((i >> np.uint64(2)) * np.uint64(0x9E3779B9)) & A.M32) ^ key)]
    for _ in range(5):
        w.append(A._next(w[-1]))
    s = np.choose((i & np.uint64(3)).astype(int), w[2:])
    cm, cv, t = A.encode(mo, vo, (s & np.uint64(0xFFFF)).astype(np.uint32),
                         (s >> np.uint64(16)).astype(np.uint32))
    assert np.array_equal(host(m[n - k:]), cm) and np.array_equal(host(v[n - k:]), cv)
    assert np.array_equal(host(tops[-(k // 256 + 1):])[-len(t):], t)
    assert float(p[:512].float().abs().min()) > 0 and float(p[600:1 << 20].float().abs().max()) == 0
    del p, g, m, v, tops, plan
    torch.cuda.empty_cache()


@pytest.mark.parametrize("param", [F, B])
@pytest.mark.parametrize("eight", [False, True])
def test_a_rate_that_is_not_a_number_shows(param, eight):
    """Every kind of NaN as the learning rate leaves NaN parameters, not zeros."""
    say("case: adamw, learning rate NaN", param, eight)
    n = 3000
    for word in (0x7FC00000, 0x7FFFFFFF, -1, 0x7FFFC001):
        rng = np.random.default_rng(106)
        p, g, m, v, tops = draw(rng, n, param, param, eight, 0)
        plan = U.adamw_prepare([p], [g], [m], [v], tops=[tops] if eight else None,
                               weight_decay=0.1)
        sched = torch.tensor([word, 0x3F800000], dtype=torch.int64).to(torch.int32)
        sched = sched.to(DEV).view(torch.float32)
        U.adamw(plan, torch.ones(1, dtype=torch.int32, device=DEV), sched, seed=3)
        assert bool(torch.isnan(p).all()), hex(word)


def busy():
    """Work on the current stream that takes some 20 ms, and no answer from the device."""
    x = torch.empty(1 << 28, device=DEV)
    for _ in range(100):
        x.fill_(1.0)


def test_a_plan_made_on_another_stream_is_whole():
    """The table of tensors outlives what the current stream still does with its memory."""
    say("case: adamw, a plan made on another stream")
    p, g, m, v = (torch.ones(5000, device=DEV) for _ in range(4))
    want = U.adamw_prepare([p], [g], [m], [v]).buf.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.empty_like(want)
    busy()
    old.fill_(7)
    old = None                                                   # freed, the fill still queued
    plan = U.adamw_prepare([p], [g], [m], [v], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(plan.buf, want)


@pytest.mark.parametrize("given", [True, False])
def test_a_plan_may_be_dropped_while_a_step_runs(given):
    """A step waits on another stream (given, or the current one then) while its plan is dropped:
    the memory of its table is not handed out again before."""
    say("case: adamw, a plan dropped while a step runs", given)
    n = 50000
    sets = [[torch.full((n,), 0.5, device=DEV) for _ in range(4)] for _ in range(2)]
    step = torch.ones(1, dtype=torch.int32, device=DEV)
    sched = torch.tensor([1e-3, 1.0], device=DEV)
    U.adamw(U.adamw_prepare(*[[x] for x in sets[0]]), step, sched)
    plan = U.adamw_prepare(*[[x] for x in sets[1]])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    where, size = plan.buf.data_ptr(), plan.buf.numel()
    with torch.cuda.stream(side):
        busy()
        if not given:
            U.adamw(plan, step, sched)
    if given:
        U.adamw(plan, step, sched, stream=side)
    plan = None
    others = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(20)]
    assert all(x.data_ptr() != where for x in others)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*sets))


@pytest.mark.parametrize("param,eight", [(B, True), (F, True), (B, False)])
def test_steps_repeat_their_bits(param, eight):
    """The same states, seed and gradients give the same bits, step after step; another seed
    gives others."""
    say("case: adamw, repeated", param, eight)
    n = 70001

    def train(seed):
        rng = np.random.default_rng(107)
        p, g, m, v, tops = draw(rng, n, param, param, eight, 0)
        plan = U.adamw_prepare([p], [g], [m], [v], tops=[tops] if eight else None,
                               weight_decay=0.1)
        step, sched = torch.zeros(1, dtype=torch.int32, device=DEV), torch.tensor([1e-3, 1.0],
                                                                                 device=DEV)
        for _ in range(6):
            step += 1
            U.adamw(plan, step, sched, seed=seed)
        return [p, m, v] + ([tops] if eight else [])

    a, b, c = train(5), train(5), train(6)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not torch.equal(a[0], c[0])


def test_bf16_copies_of_every_parameter():
    """All 2^32 words as parameters, a step that changes none (signalling NaNs become quiet): the
    copy is the nearest bf16, ties to even, a NaN its upper half."""
    say("case: adamw, bf16 copies of every word")
    n = 1 << 28
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of device memory")
    g = torch.zeros(n, device=DEV)
    p, copy = torch.empty(n, device=DEV), torch.empty(n, dtype=B, device=DEV)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    plan = U.adamw_prepare([p], [g], [m], [v], copies=[copy])
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    sched = torch.tensor([0.0, 1.0], device=DEV)
    for k in range(16):
        word = torch.arange(n, dtype=torch.int32, device=DEV) + (k - 8) * n
        p.view(torch.int32).copy_(word)
        U.adamw(plan, one, sched)
        nan = (word & 0x7FFFFFFF) > 0x7F800000
        word = torch.where(nan, word | 0x400000, word)
        assert torch.equal(p.view(torch.int32), word), k
        near = torch.where(nan, word, word + 0x7FFF + ((word >> 16) & 1)) >> 16
        assert torch.equal(copy.view(torch.int16), near.to(torch.int16)), k
    del g, p, copy, m, v, plan, word, nan, near
    torch.cuda.empty_cache()
