"""GPU parity of the rows in 8 bits and of the experts' products on them.

Integers and scales of rows are compared for equality.  A product's integer sum is exact; turning
it into fp32 and its two scales round three times (3 eps, eps = 2^-24), the store by half a bf16 step
(2^-8 of the value).  SwiGLU: with a gate g off by 3 eps, e^-g is off by (3 |g| + |g| + 2) eps (its
argument rounded once, exp2 two units), 1 + e^-g, the reciprocal and three products add 7, the
up value 3: within (4 |g| + 16) eps, then the store."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle as O                                       # noqa: E402
from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, to_dev, host, say, err_word, random_routing   # noqa: E402
from tests.test_gpu_combine import oracle_dest_row       # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------- rows
def awkward_rows(n, H, seed):
    """bf16 rows of every size: wide, tiny, zero, subnormal, and full of quotients at a border."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, H, generator=g, device=DEV)
    x *= 10.0 ** torch.randint(-3, 4, (n, 1), generator=g, device=DEV)
    if n > 8:
        x[1] = 0
        x[2] *= 1e-38
        x[3] *= 1e36
        x[4] = torch.randint(-254, 255, (H,), generator=g, device=DEV) * 0.5    # ties
        x[4, 0] = 127.0
        x[5] = 0
        x[5, H - 1] = -3e38
        x[6] = 1e-40
        x[7] = -x[7].abs()
        x[8] = torch.randint(-254, 255, (H,), generator=g, device=DEV) * 0.5 * 0.0078125
        x[8, 1] = 127.0 * 0.0078125
    return x.to(torch.bfloat16)


def flag(x):
    """A row of the widest range may hold an infinity."""
    return 0 if bool(torch.isfinite(x).all()) else U.ERR_VALUE


@pytest.mark.parametrize("n,H", [(1, 16), (3, 32), (20, 48), (1, 4096), (37, 1024), (33, 1040),
                                 (21, 2048), (20, 4112), (19, 7168), (17, 8192), (18, 16384),
                                 (11, 16400), (10, 40000), (9, 65536), (5000, 256)])
def test_rows(n, H):
    say("case: rows", n, H)
    x, err = awkward_rows(n, H, n + H), err_word()
    q, s = U.quant_rows(x, err=err)
    q_o, s_o = O.quant_rows(f64(x))
    assert int(host(err)[0]) == flag(x)
    assert np.array_equal(host(s), s_o) and np.array_equal(host(q), q_o)


@pytest.mark.parametrize("H", [16, 1024, 7168])
def test_every_bf16_value_against_every_border(H):
    """All finite bf16 numbers up to a row's maximum, for maxima that put quotients close to
    borders: integers as the 64-bit quotient says."""
    say("case: all values", H)
    bits = np.arange(0x7F80, dtype=np.uint32)
    vals = (bits << 16).view(np.float32)
    for top in (1.0, 1.0078125, 126.5, 127.0, 1.9921875, 3.0, 2.0 ** 100 * 1.25, 2.0 ** -118):
        v = np.concatenate([vals[vals <= top], -vals[vals <= top]])
        v = v[np.abs(v) >= top / 600]                 # smaller ones are 0 for sure
        n = -(-len(v) // (H - 1))
        x = np.zeros((n, H), np.float32)
        x[:, 1:].reshape(-1)[:0] = 0
        flat = np.zeros(n * (H - 1), np.float32)
        flat[:len(v)] = v
        x[:, 1:] = flat.reshape(n, H - 1)
        x[:, 0] = top
        xd = to_dev(x, torch.bfloat16)
        q, s = U.quant_rows(xd)
        q_o, s_o = O.quant_rows(f64(xd))
        assert np.array_equal(host(s), s_o) and np.array_equal(host(q), q_o), top


@pytest.mark.parametrize("H", [16, 1024, 5008, 20000])
def test_rows_that_are_not_numbers(H):
    x = awkward_rows(12, H, 1)
    x[0, 3], x[2, 5], x[9, 7], x[10] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[11, :] = float("inf")
    err = err_word()
    q, s = U.quant_rows(x, err=err)
    q_o, s_o = O.quant_rows(f64(x))
    assert int(host(err)[0]) == U.ERR_VALUE
    assert np.array_equal(host(s), s_o) and np.array_equal(host(q), q_o)


@pytest.mark.parametrize("live", [-3, 0, 1, 17, 40, 1000])
@pytest.mark.parametrize("H", [64, 2064])
def test_rows_behind_the_live_ones_stay(H, live):
    x = awkward_rows(40, H, 5)
    x[39, 0] = float("nan")                            # not read where it is not live
    q = torch.full((40, H), 99, dtype=torch.int8, device=DEV)
    s = torch.full((40,), 99.0, device=DEV)
    err = err_word()
    U.quant_rows(x, q, s, live_rows=torch.tensor([live], dtype=torch.int32, device=DEV), err=err)
    q_o, s_o = O.quant_rows(f64(x))
    n = min(max(live, 0), 40)
    assert np.array_equal(host(q)[:n], q_o[:n]) and np.array_equal(host(s)[:n], s_o[:n])
    assert (host(q)[n:] == 99).all() and (host(s)[n:] == 99).all()
    assert int(host(err)[0]) == flag(x[:n])


@pytest.mark.parametrize("R,T,K,E,H,empty", [
    (4, 128, 2, 8, 256, 0.0), (3, 47, 3, 9, 2064, 0.1), (1, 1, 8, 16, 4096, 0.0),
    (2, 9, 20, 24, 48, 0.3), (1, 5, 4, 8, 40000, 0.2), (1, 3, 64, 64, 16, 0.0),
    (2, 300, 1, 4, 7168, 0.5)])
def test_dispatch(R, T, K, E, H, empty):
    say("case: dispatch in 8 bits", R, T, K, E, H, empty)
    rng = np.random.default_rng(H + T)
    dr = oracle_dest_row(random_routing(rng, R, T, K, E, empty_frac=empty), E, 1, 2)
    P = int((dr >= 0).sum()) + 3
    x = awkward_rows(R * T, H, T).view(R, T, H)
    q = torch.full((P, H), 99, dtype=torch.int8, device=DEV)
    s = torch.full((P,), 99.0, device=DEV)
    err = err_word()
    U.permute_quant(x, to_dev(dr), q, s, err=err)
    q_o, s_o = O.quant_rows(f64(x))
    want_q, want_s = np.full((P, H), 99, np.int8), np.full(P, 99, np.float32)
    for k in range(K):
        r, t = np.nonzero(dr[..., k] >= 0)
        want_q[dr[r, t, k]], want_s[dr[r, t, k]] = q_o[r, t], s_o[r, t]
    assert int(host(err)[0]) == flag(x[torch.from_numpy((dr >= 0).any(-1)).to(DEV)])
    err.zero_()
    assert np.array_equal(host(q), want_q) and np.array_equal(host(s), want_s)
    # some ranks only; rows outside of the buffer are skipped and flagged
    q.fill_(99), s.fill_(99)
    U.permute_quant(x, to_dev(dr), q, s, r_begin=R - 1)
    own = dr[R - 1][dr[R - 1] >= 0]
    other = np.setdiff1d(np.arange(P), own)
    assert np.array_equal(host(q)[own], want_q[own]) and (host(q)[other] == 99).all()
    assert np.array_equal(host(s)[own], want_s[own]) and (host(s)[other] == 99).all()
    bad = dr.copy()
    bad[0, 0, 0], bad[R - 1, T - 1, K - 1] = P, -2
    q.fill_(99), s.fill_(99)
    U.permute_quant(x, to_dev(bad), q, s, err=err)
    keep = np.ones(P, bool)
    keep[[d for d in (dr[0, 0, 0], dr[R - 1, T - 1, K - 1]) if d >= 0]] = False
    assert int(host(err)[0]) & ~U.ERR_VALUE == U.ERR_ROW_RANGE
    assert np.array_equal(host(q)[keep], want_q[keep]) and (host(q)[~keep] == 99).all()


def test_dispatch_into_no_rows():
    x, err = awkward_rows(9, 32, 1).view(1, 9, 32), err_word()
    q, s = torch.empty(0, 32, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV)
    row = torch.full((1, 9, 2), -1, dtype=torch.int32, device=DEV)
    U.permute_quant(x, row, q, s, err=err)
    assert int(host(err)[0]) == 0
    row[0, 4, 1] = 0
    U.permute_quant(x, row, q, s, err=err)
    assert int(host(err)[0]) == U.ERR_ROW_RANGE             # before its row is read


# ----------------------------------------------------------------------------- products
def operands(rows, R, E, S, N, D, seed, full=False):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def codes(*shape):
        if full:                                       # -128 and 127 throughout
            return (torch.randint(0, 2, shape, generator=g, device=DEV) * 255 - 128).to(torch.int8)
        return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)

    def scales(*shape):
        return (0.5 + torch.rand(shape, generator=g, device=DEV)) / (40.0 * D ** 0.5)

    return dict(q=codes(rows, D), q_scale=scales(rows) * 2, w=codes(E, N, D), w_scale=scales(E, N),
                slot_w=codes(R, S, N, D) if S else None,
                slot_scale=scales(R, S, N) if S else None)


def blocks(rng, rows, n_inst, lead=0, tail=0, even=False):
    """Offsets of n_inst instances over the rows, some empty, some rows before and behind."""
    live = rows - lead - tail
    if even:
        cut = np.linspace(0, live, n_inst + 1).astype(int)
    else:
        p = rng.dirichlet(np.full(n_inst, 0.5))
        cut = np.concatenate([[0], np.cumsum(rng.multinomial(live, p))])
    return (cut + lead).astype(np.int32)


def run_product(o, off, R, S, act, out, err=None, stream=None):
    return U.expert_product(o["q"], o["q_scale"], o["w"], o["w_scale"],
                            inst_offset=None if off is None else to_dev(off), R=R, S=S,
                            slot_w=o["slot_w"], slot_scale=o["slot_scale"], act=act, out=out,
                            err=err, stream=stream)


def check_product(o, off, R, E, S, act, out, fill):
    rows = out.shape[0]
    h = {k: None if v is None else host(v) for k, v in o.items()}
    table = [0, rows] if off is None else off
    got, seen = f64(out), np.zeros(rows, bool)
    for at, y, gate in O.expert_product(h["q"], h["q_scale"], table, R, E, S, h["w"], h["w_scale"],
                                        h["slot_w"], h["slot_scale"], act == U.PRODUCT_SWIGLU):
        units = 3 if gate is None else 4 * np.abs(gate) + 16
        room = units * EPS * np.abs(y)
        assert (np.abs(got[at] - y) <= room + 2.0 ** -8 * (np.abs(y) + room) + 2.0 ** -133).all()
        seen[at] = True
    assert (got[~seen] == fill).all()                  # rows of no instance


# rows, R, E, S, N, D
SHAPES = [
    (1, 1, 1, 0, 16, 16), (1, 1, 1, 0, 4096, 512), (5, 1, 1, 0, 48, 48), (16, 1, 1, 0, 64, 64),
    (17, 1, 1, 0, 16, 4112), (64, 1, 1, 0, 256, 256), (65, 1, 1, 0, 272, 336),
    (300, 1, 1, 0, 512, 1040), (8, 1, 32, 0, 128, 640), (40, 2, 8, 1, 96, 176),
    (200, 4, 8, 2, 80, 272), (1000, 2, 6, 1, 144, 208), (900, 1, 3, 0, 528, 400),
    (2500, 1, 2, 0, 1024, 512), (3000, 2, 4, 1, 320, 1168), (1500, 1, 5, 0, 1008, 128),
    (33, 64, 256, 8, 16, 32),
    # one of each of the call's forms at the least, with edges of tiles inside of everything
    (5003, 1, 7, 0, 2576, 272),        # 256 x 256, several tiles a workgroup, half-empty ones
    (9000, 1, 3, 0, 1040, 144),        # 256 x 256, two steps
    (2100, 2, 4, 0, 2064, 400), (1000, 1, 1, 0, 4080, 4112),       # 128 x 128, two and one a CU
    (1000, 1, 4, 0, 1040, 4112), (250, 1, 1, 0, 4080, 4112),       # 64 x 128, 64 x 64
    (1100, 4, 16, 1, 2064, 528), (120, 1, 1, 0, 4080, 4112),       # 128 x 64, 64 x 32 (depth in 2)
    (60, 4, 16, 1, 2064, 528), (60, 1, 1, 0, 4080, 4112),          # 64 x 32, 32 x 32
    (30, 1, 1, 0, 4080, 4112), (16, 1, 1, 0, 4080, 7184),          # 32 x 16; 16 x 16, SwiGLU 32 x 16
    (40, 2, 8, 1, 272, 4112),          # the same, several instances, a ragged last round of steps
    (3, 1, 1, 0, 1 << 20, 16),         # very wide
]


@pytest.mark.parametrize("act", [U.PRODUCT_PLAIN, U.PRODUCT_SWIGLU])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(shape, act):
    say("case: product", *shape, act)
    rows, R, E, S, N, D = shape
    rng = np.random.default_rng(rows + N)
    o = operands(rows, R, E, S, N, D, rows + N + D)
    n_inst = R * (E // R + S)
    lead, tail = (0, 0) if rows < 20 else (3, 5)
    off = None if n_inst == 1 else blocks(rng, rows, n_inst, lead, tail)
    n_out = N // 2 if act == U.PRODUCT_SWIGLU else N
    out = torch.full((rows, n_out), 7.0, dtype=torch.bfloat16, device=DEV)
    err = err_word()
    run_product(o, off, R, S, act, out, err)
    assert int(host(err)[0]) == 0
    check_product(o, off, R, E, S, act, out, 7.0)
    again = torch.full_like(out, 7.0)
    run_product(o, off, R, S, act, again)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_sums_at_the_ends_of_the_range():
    """Integers of -128 and 127 over the longest depth: sums up to 2^30 are exact."""
    say("case: product, largest sums")
    o = operands(20, 1, 1, 0, 16, 65536, 3, full=True)
    o["q"][0], o["w"][0, 0] = -128, -128               # 2^30
    o["q"][1], o["w"][0, 1] = 127, -128
    out = torch.empty(20, 16, dtype=torch.bfloat16, device=DEV)
    run_product(o, None, 1, 0, U.PRODUCT_PLAIN, out)
    check_product(o, None, 1, 1, 0, U.PRODUCT_PLAIN, out, 0.0)


def test_scales_far_apart():
    """Scales whose own product leaves the range, with results in it."""
    o = operands(8, 1, 1, 0, 16, 64, 4)
    o["q_scale"][:] = torch.tensor([1e30, 1e-30, 2.0 ** -126, 0.0, 1e-20, 1e20, 1.0, 1e10])
    out = torch.empty(8, 16, dtype=torch.bfloat16, device=DEV)
    run_product(o, None, 1, 0, U.PRODUCT_PLAIN, out)
    check_product(o, None, 1, 1, 0, U.PRODUCT_PLAIN, out, 0.0)


def test_every_instance_empty_or_one_has_all():
    o = operands(70, 2, 4, 1, 32, 64, 5)
    out = torch.full((70, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    run_product(o, np.full(7, 9, np.int32), 2, 1, U.PRODUCT_PLAIN, out)
    assert (f64(out) == 7).all()
    for i in range(6):
        off = np.where(np.arange(7) <= i, 0, 70).astype(np.int32)
        run_product(o, off, 2, 1, U.PRODUCT_PLAIN, out)
        check_product(o, off, 2, 4, 1, U.PRODUCT_PLAIN, out, 7.0)
    empty = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    none = dict(o, q=o["q"][:0], q_scale=o["q_scale"][:0])
    run_product(none, np.zeros(7, np.int32), 2, 1, U.PRODUCT_PLAIN, empty)


@pytest.mark.parametrize("off", [[0, 50, 20, 100], [-5, 10, 20, 100], [0, 10, 20, 300],
                                 [90, 60, 30, 0], [2 ** 31 - 1] * 4, [-2 ** 31] * 4])
def test_bad_offsets_are_flagged(off):
    say("case: product, bad offsets", off)
    for rows_per in (100, 1):                          # few and many rows an instance
        o = operands(100, 1, 3, 0, 32, 128, 6)
        guard = torch.full((300, 32), 7.0, dtype=torch.bfloat16, device=DEV)
        err = err_word()
        run_product(o, np.array(off, np.int32), 1, 0, U.PRODUCT_PLAIN, guard[100:200], err)
        assert int(host(err)[0]) == U.ERR_OFFSET
        assert (f64(guard[:100]) == 7).all() and (f64(guard[200:]) == 7).all()


@pytest.mark.parametrize("rows", [400, 3000, 20000])
def test_offsets_that_name_rows_many_times(rows):
    """A table that goes up and down names far more tiles than its rows make: flagged, and no more
    of them worked on than the rows could make."""
    say("case: product, rising and falling offsets", rows)
    o = operands(rows, 1, 200, 0, 2048, 32, 7)
    off = np.tile(np.array([0, rows], np.int32), 101)[:201]
    guard = torch.full((rows + 200, 2048), 7.0, dtype=torch.bfloat16, device=DEV)
    err = err_word()
    run_product(o, off, 1, 0, U.PRODUCT_PLAIN, guard[100:-100], err)
    assert int(host(err)[0]) == U.ERR_OFFSET
    assert (f64(guard[:100]) == 7).all() and (f64(guard[-100:]) == 7).all()


@pytest.mark.parametrize("rows,N,D,act", [(1, 1000, 1040, 0), (5, 264, 336, 0), (33, 1008, 4112, 1),
                                          (300, 4104, 144, 0), (700, 2064, 1040, 1),
                                          (5000, 2056, 272, 0), (5000, 2064, 144, 1)])
def test_operands_at_the_end_of_their_memory(rows, N, D, act):
    """Rows, weights and scales behind which nothing that could be read is the same: the result
    does not depend on what follows them in memory, in partial tiles of every kind."""
    say("case: product, ends of memory", rows, N, D, act)
    o = operands(rows, 1, 1, 0, N, D, 12)
    n_out = N // 2 if act else N
    outs = []
    for fill in (0, 85):
        tail = {}
        for k in ("q", "q_scale", "w", "w_scale"):
            t = o[k]
            flat = torch.full((t.numel() * t.element_size() + 65536,), fill, dtype=torch.uint8,
                              device=DEV)
            flat[:t.numel() * t.element_size()] = t.reshape(-1).view(torch.uint8)
            tail[k] = flat[:t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        out = torch.full((rows + 300, n_out), 7.0, dtype=torch.bfloat16, device=DEV)
        run_product(dict(o, **tail), None, 1, 0, act, out[:rows])
        assert (f64(out[rows:]) == 7).all()
        outs.append(out[:rows].clone())
    assert torch.equal(outs[0], outs[1])
    check_product(o, None, 1, 1, 0, act, outs[0], 7.0)


def test_row_offsets_past_32_bits():
    """Rows and outputs of more than 2^31 and 2^32 bytes: the last block against its own product."""
    say("case: product, long buffers")
    rows, D, N = 140000, 16384, 64
    q = torch.empty(rows, D, dtype=torch.int8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(8)
    q.fill_(1)
    q[-300:] = torch.randint(-127, 128, (300, D), generator=g, device=DEV, dtype=torch.int8)
    o = operands(300, 1, 2, 0, N, D, 8)
    long = dict(o, q=q, q_scale=torch.full((rows,), 1e-3, device=DEV))
    long["q_scale"][-300:] = o["q_scale"]
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    run_product(long, np.array([0, rows - 300, rows], np.int32), 1, 0, U.PRODUCT_PLAIN, out)
    short = torch.zeros(300, N, dtype=torch.bfloat16, device=DEV)
    run_product(dict(o, q=q[-300:].contiguous()), np.array([0, 0, 300], np.int32), 1, 0,
                U.PRODUCT_PLAIN, short)
    assert torch.equal(out[-300:], short)
    want = (o["w"][0].double().sum(-1) * o["w_scale"][0].double() * float(np.float32(1e-3))).cpu().numpy()
    got = f64(out[[0, 70000, rows - 301]])
    assert (np.abs(got - want) <= (2.0 ** -8 + 8 * EPS) * np.abs(want)).all()


def test_captured_and_replayed_on_a_stream():
    """The expert path in 8 bits in one graph, replayed on new rows and a new plan."""
    say("case: product, captured")
    g = torch.Generator(device=DEV).manual_seed(9)
    R, E, S, T, K, H, F = 2, 4, 1, 60, 2, 128, 64
    o1, o2 = operands(1, R, E, S, 2 * F, H, 10), operands(1, R, E, S, H, F, 11)
    x = torch.zeros(R, T, H, dtype=torch.bfloat16, device=DEV)
    drow = torch.full((R, T, K), -1, dtype=torch.int32, device=DEV)
    off = torch.zeros(R * 3 + 1, dtype=torch.int32, device=DEV)
    P = R * T * K
    q, s = torch.zeros(P, H, dtype=torch.int8, device=DEV), torch.zeros(P, device=DEV)
    q2, s2 = torch.zeros(P, F, dtype=torch.int8, device=DEV), torch.zeros(P, device=DEV)
    h = torch.zeros(P, F, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(P, H, dtype=torch.bfloat16, device=DEV)
    err = err_word()

    def path():
        U.permute_quant(x, drow, q, s, err=err)
        U.expert_product(q, s, o1["w"], o1["w_scale"], off, R, S, o1["slot_w"], o1["slot_scale"],
                         U.PRODUCT_SWIGLU, h, err)
        U.quant_rows(h, q2, s2, live_rows=off[-1:], err=err)
        U.expert_product(q2, s2, o2["w"], o2["w_scale"], off, R, S, o2["slot_w"],
                         o2["slot_scale"], out=out, err=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        path()
        with torch.cuda.graph(graph, stream=side):
            path()
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(torch.randn(R, T, H, generator=g, device=DEV))
        ids = torch.topk(torch.randn(R, T, E, generator=g, device=DEV), K, -1).indices.to(torch.int32)
        plan = U.plan(ids, E, S, 4)
        drow.copy_(plan["dest_row"]), off.copy_(plan["inst_offset"])
        for t in (q, s, q2, s2, h, out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, s, h, q2, s2, out)]
        for t in (q, s, q2, s2, h, out):
            t.zero_()
        path()
        assert all(torch.equal(a, b) for a, b in zip(got, (q, s, h, q2, s2, out)))
        o = dict(o2, q=q2, q_scale=s2)
        check_product(o, host(off), R, E, S, U.PRODUCT_PLAIN, out, 0.0)
    assert int(host(err)[0]) == 0


def test_binding_refusals():
    bf, i8 = torch.bfloat16, torch.int8
    x = torch.zeros(4, 32, dtype=bf, device=DEV)
    q, s = U.quant_rows(x)
    w, ws = torch.zeros(2, 16, 32, dtype=i8, device=DEV), torch.ones(2, 16, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    row = torch.zeros(1, 4, 1, dtype=torch.int32, device=DEV)
    for call in (
            lambda: U.quant_rows(x.half()), lambda: U.quant_rows(x.float()),
            lambda: U.quant_rows(x[0]), lambda: U.quant_rows(x, q=q[:3]),
            lambda: U.quant_rows(x, q=q.view(torch.uint8)), lambda: U.quant_rows(x, scale=s[:3]),
            lambda: U.quant_rows(x.cpu()), lambda: U.quant_rows(x.t()),
            lambda: U.permute_quant(x, row, q, s),
            lambda: U.permute_quant(x[None], row, q, s[:2]),
            lambda: U.permute_quant(x[None], row, q[:, :16], s),
            lambda: U.permute_quant(x[None], row[:, :2].contiguous(), q, s),
            lambda: U.expert_product(q, s, w.float(), ws, off),
            lambda: U.expert_product(q[:, :16], s, w, ws, off),
            lambda: U.expert_product(q, s[:2], w, ws, off),
            lambda: U.expert_product(q, s, w, ws[:1], off),
            lambda: U.expert_product(q, s, w, ws, off[:2]),
            lambda: U.expert_product(q, s, w, ws, off, S=1, slot_w=w[:0], slot_scale=ws),
            lambda: U.expert_product(q, s, w, ws, off, out=torch.zeros(4, 8, dtype=bf, device=DEV))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: U.quant_rows(x[:, :24].contiguous()),
                 lambda: U.expert_product(q, s, w, ws),
                 lambda: U.expert_product(q, s, w, ws, off, act=5),
                 lambda: U.expert_product(q, s, w, ws, torch.zeros_like(row).view(4), S=1)):
        with pytest.raises(U.UEPError):
            call()
