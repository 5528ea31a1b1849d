"""GPU parity of uep_permute_grad and uep_combine_grad against the oracle: dx and dout bit
for bit; the weights' gradient against a 64-bit sum, to (H / 64 + 16) eps = 2^-24 of the
sum of magnitudes (products of two bf16 are exact in fp32; a lane adds at most H / 64 + 7
of them one after the other, and the lanes' sums and slices add a few more)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle as O                                       # noqa: E402
from moe_expert_load_amd import uep as U                 # noqa: E402
from tests.gpu_helpers import DEV, to_dev, host, say, err_word, random_routing  # noqa: E402
from tests.test_gpu_combine import bits, oracle_dest_row  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24

CASES = [
    (0, 4, 512, 2, 8, 256, 0.0),          # tiny shape
    (1, 3, 97, 3, 9, 8 * 300, 0.1),       # ragged slices
    (2, 2, 40, 5, 10, 7168, 0.2),         # 14 KiB rows, empty slots
    (3, 5, 33, 9, 15, 1032, 0.05),        # K = 9, odd row length
    (4, 1, 64, 1, 1, 64, 0.3),            # one rank, one expert
    (5, 1, 1, 8, 16, 4096, 0.0),          # one token
    (6, 1, 3, 2, 4, 8, 0.0),              # the shortest rows
    (7, 1, 7, 20, 24, 520, 0.1),          # many slots
    (8, 2, 5, 4, 8, 16392, 0.3),          # rows longer than any slice
    (9, 1, 2, 8, 8, 4096, 0.9),           # nearly everything empty
]


def make(seed, R, T, K, E, H, empty, extra=0):
    rng = np.random.default_rng(seed)
    ids = random_routing(rng, R, T, K, E, empty_frac=empty)
    dr = oracle_dest_row(ids, E, 1, 2)
    P = max(int((dr >= 0).sum()), 1) + extra
    g = torch.Generator(device=DEV).manual_seed(seed)
    dy = torch.randn(R, T, H, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.randn(P, H, generator=g, device=DEV).to(torch.bfloat16)
    w = rng.random((R, T, K)).astype(np.float32) * 2 - 0.5
    return dr, dy, out, w


@pytest.mark.parametrize("case", CASES)
def test_permute_grad(case):
    say("case: permute_grad", *case)
    dr, dy, out, _ = make(*case)
    dx = torch.full(dy.shape, 77, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    U.permute_grad(out, to_dev(dr), dx)
    assert np.array_equal(bits(dx), O.permute_grad(bits(out), dr))


@pytest.mark.parametrize("case", CASES)
def test_combine_grad(case):
    say("case: combine_grad", *case)
    dr, dy, out, w = make(*case, extra=3)
    P, H = out.shape
    fill = torch.full((P, H), 77, dtype=torch.int16, device=DEV)
    dout, dw = fill.clone().view(torch.bfloat16), torch.full(w.shape, 9.0, device=DEV)
    err = err_word()
    drow, wd = to_dev(dr), to_dev(w, torch.float32)
    U.combine_grad(dy, out, drow, wd, dout, dw, err=err)
    dout_o, dw_o, mag = O.combine_grad(bits(dy), bits(out), dr, w)
    named = np.zeros(P, bool)
    named[dr[dr >= 0]] = True
    assert int(host(err)[0]) == 0
    assert np.array_equal(bits(dout)[named], dout_o[named])
    assert (bits(dout)[~named] == 77).all()                       # rows without a slot
    assert (np.abs(host(dw) - dw_o) <= (H / 64 + 16) * EPS * mag).all()
    assert (host(dw)[dr < 0] == 0).all()
    # the same bits again, only dout without the weights' gradient, and in place
    dw2, only, place = torch.empty_like(dw), fill.clone().view(torch.bfloat16), out.clone()
    U.combine_grad(dy, out, drow, wd, dout, dw2)
    assert torch.equal(dw, dw2)
    U.combine_grad(dy, None, drow, wd, only)
    assert np.array_equal(bits(only), bits(dout))
    U.combine_grad(dy, place, drow, wd, place, dw2)
    assert torch.equal(dw, dw2)
    assert np.array_equal(bits(place)[named], dout_o[named])
    assert np.array_equal(bits(place)[~named], bits(out)[~named])


@pytest.mark.parametrize("R,T,K,H", [
    (3, 4000, 4, 1032),       # 99 MB of rows: two phases, one chunk, a rank range
    (2, 15000, 2, 4096),      # 246 MB of gradients: two chunks
    (1, 100, 8, 40000),       # few tokens, long rows, in phases
])
def test_combine_grad_in_phases(R, T, K, H):
    """Large calls run the dot products and the scaled rows apart.  The reference is torch on
    the device: one fp32 product rounded to bf16, and the dot products in 64 bits."""
    say("case: combine_grad in phases", R, T, K, H)
    g = torch.Generator(device=DEV).manual_seed(R * T)
    n = R * T * K
    row = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    row[torch.rand(n, generator=g, device=DEV) < 0.05] = -1
    row = row.view(R, T, K)
    dy = torch.randn(R, T, H, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.randn(n, H, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.rand(R, T, K, generator=g, device=DEV)
    for lo, hi in ((0, R), (R - 1, R)):
        dout = torch.full((n, H), 77, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        dw = torch.full((R, T, K), 9.0, device=DEV)
        place, dw2 = out.clone(), torch.empty_like(dw)
        U.combine_grad(dy, out, row, w, dout, dw, r_begin=lo, r_end=hi)
        U.combine_grad(dy, place, row, w, place, dw2, r_begin=lo, r_end=hi)
        for k in range(K):
            d = row[lo:hi, :, k].reshape(-1)
            on = d >= 0
            rows, grad = d[on].long(), dy[lo:hi].reshape(-1, H)[on]
            want = (w[lo:hi, :, k].reshape(-1)[on, None] * grad.float()).to(torch.bfloat16)
            assert torch.equal(dout[rows].view(torch.int16), want.view(torch.int16))
            assert torch.equal(place[rows].view(torch.int16), want.view(torch.int16))
            got = dw[lo:hi, :, k].reshape(-1)
            dot = torch.cat([(grad[a:a + 2000].double() * out[rows[a:a + 2000]].double()).sum(-1)
                             for a in range(0, len(rows), 2000)])
            mag = torch.cat([(grad[a:a + 2000].double() * out[rows[a:a + 2000]].double()).abs()
                             .sum(-1) for a in range(0, len(rows), 2000)])
            assert ((got[on].double() - dot).abs() <= (H / 64 + 16) * EPS * mag).all()
            assert (got[~on] == 0).all()
        assert torch.equal(dw[lo:hi], dw2[lo:hi]) and (dw[:lo] == 9).all()
        named = torch.zeros(n, dtype=torch.bool, device=DEV)
        named[row[lo:hi][row[lo:hi] >= 0].long()] = True
        assert (dout.view(torch.int16)[~named] == 77).all()
        assert torch.equal(place.view(torch.int16)[~named], out.view(torch.int16)[~named])


def test_rank_ranges_and_noops():
    say("case: row gradients, rank ranges")
    dr, dy, out, w = make(11, 4, 50, 4, 8, 512, 0.1)
    drow, wd = to_dev(dr), to_dev(w, torch.float32)
    fill = torch.full(dy.shape, 77, dtype=torch.int16, device=DEV)
    dx = fill.clone().view(torch.bfloat16)
    U.permute_grad(out, drow, dx, r_begin=1, r_end=3)
    want = O.permute_grad(bits(out), dr)
    assert np.array_equal(bits(dx)[1:3], want[1:3]) and (bits(dx)[[0, 3]] == 77).all()
    dout = torch.full(out.shape, 77, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    dw = torch.full(w.shape, 9.0, device=DEV)
    U.combine_grad(dy, out, drow, wd, dout, dw, r_begin=2, r_end=3)
    dout_o, dw_o, _ = O.combine_grad(bits(dy), bits(out), dr, w)
    mine = dr[2][dr[2] >= 0]
    assert np.array_equal(bits(dout)[mine], dout_o[mine])
    rest = np.setdiff1d(np.arange(out.shape[0]), mine)
    assert (bits(dout)[rest] == 77).all() and (host(dw)[[0, 1, 3]] == 9).all()
    U.combine_grad(dy, out, drow, wd, dout, dw, r_begin=1, r_end=1)
    assert (host(dw)[[0, 1, 3]] == 9).all()
    none = to_dev(np.full(dr.shape, -1))
    U.permute_grad(out, none, dx)
    assert (bits(dx) == 0).all()
    U.combine_grad(dy, out, none, wd, dout, dw)
    assert (host(dw) == 0).all()


def test_rows_outside_the_buffer_are_flagged():
    say("case: row gradients, rows out of range")
    dr, dy, out, w = make(12, 2, 30, 3, 6, 264, 0.0)
    P = out.shape[0]
    bad = dr.copy()
    bad[0, 0, 0], bad[1, 5, 2], bad[1, 29, 1] = P, 2 ** 31 - 1, -9
    ok = np.where((bad < -1) | (bad >= P), -1, bad)
    e1, e2 = err_word(), err_word()
    dx, dout = torch.empty_like(dy), torch.zeros_like(out)
    U.permute_grad(out, to_dev(bad), dx, err=e1)
    _, dw = U.combine_grad(dy, out, to_dev(bad), to_dev(w, torch.float32), dout, err=e2)
    assert int(host(e1)[0]) == int(host(e2)[0]) == U.ERR_ROW_RANGE
    assert np.array_equal(bits(dx), O.permute_grad(bits(out), ok))
    dout_o, dw_o, mag = O.combine_grad(bits(dy), bits(out), ok, w)
    assert np.array_equal(bits(dout), dout_o)
    assert (np.abs(host(dw) - dw_o) <= (264 / 64 + 16) * EPS * mag).all()


def test_infinities_and_nan_stay_in_their_rows():
    say("case: row gradients, special values")
    dr, dy, out, w = make(13, 1, 20, 2, 4, 64, 0.0)
    dy[0, 3, 5], dy[0, 4, 0] = float("inf"), float("nan")
    out[dr[0, 7, 1], 2] = float("nan")
    dout = torch.empty_like(out)
    _, dw = U.combine_grad(dy, out, to_dev(dr), to_dev(w, torch.float32), dout)
    dout_o, _, _ = O.combine_grad(bits(dy), bits(out), dr, w)
    a, b = host(dout.float()), O.bf16_bits_to_f32(dout_o)
    assert np.array_equal(np.isnan(a), np.isnan(b))
    assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])
    hot = np.zeros((20, 2), bool)
    hot[3], hot[4], hot[7, 1] = True, True, True
    assert np.array_equal(~np.isfinite(host(dw)[0]), hot)


def test_gradients_match_torchs_autograd():
    """The whole chain x -> permute -> scale -> combine against torch in float64: the
    library's dx and dgate_w are those of the same function, to the bf16 steps between (three
    roundings of 2^-8 each, relative to sums of magnitudes)."""
    say("case: row gradients against autograd")
    dr, dy, _, w = make(14, 2, 60, 4, 8, 128, 0.1)
    R, T, K = dr.shape
    P = int((dr >= 0).sum())
    x = torch.randn(R, T, 128, device=DEV).to(torch.bfloat16)
    drow, wd = to_dev(dr), to_dev(w, torch.float32)
    disp = torch.zeros(P, 128, dtype=torch.bfloat16, device=DEV)
    U.permute(x, drow, disp)
    dout = torch.empty_like(disp)
    _, dw = U.combine_grad(dy, disp, drow, wd, dout)
    dx = torch.empty_like(x)
    U.permute_grad(dout, drow, dx)
    xa = x.double().cpu().requires_grad_()
    wa = torch.from_numpy(w).double().requires_grad_()
    on = torch.from_numpy((dr >= 0).astype(np.float64))
    y = ((wa * on).sum(-1, keepdim=True)) * xa              # every copy of a token is the token
    (y * dy.double().cpu()).sum().backward()
    mag = ((wa.abs() * on).sum(-1, keepdim=True) * dy.double().cpu().abs()).detach().numpy()
    assert (np.abs(host(dx.double()) - xa.grad.numpy()) <= 3 * 2.0 ** -8 * mag + 1e-30).all()
    m2 = (xa.detach().abs() * dy.double().cpu().abs()).sum(-1, keepdim=True).numpy()
    assert (np.abs(host(dw) - wa.grad.numpy()) <= 18 * EPS * m2).all()


def test_combine_grad_of_one_slot_and_many_tokens():
    """K = 1 and 2^26 + 5 tokens: more than one launch holds."""
    n, H = 2 ** 26 + 5, 8
    say("case: combine_grad, K = 1, 2^26 + 5 tokens")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    g = torch.Generator(device=DEV).manual_seed(15)
    dy = torch.randn(1, n, H, generator=g, device=DEV, dtype=torch.bfloat16)
    out = torch.randn(n, H, generator=g, device=DEV, dtype=torch.bfloat16)
    row = torch.arange(n - 1, -1, -1, device=DEV, dtype=torch.int32).view(1, n, 1)
    row[0, ::1000] = -1
    w = torch.rand(1, n, 1, generator=g, device=DEV)
    dout = torch.full((n, H), 77, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    dout, dw = U.combine_grad(dy, out, row, w, dout)
    on = row[0] >= 0                                             # [n][1]
    want = torch.where(on, (w[0] * dy[0].float()).to(torch.bfloat16).view(torch.int16), 77)
    assert torch.equal(dout.flip(0).view(torch.int16), want)
    del want, dout
    terms = dy[0].float() * out.flip(0).float()                  # exact
    dot = torch.where(on, terms.double().sum(-1, keepdim=True), 0)
    bound = (H / 64 + 16) * EPS * terms.abs().sum(-1, keepdim=True)
    assert bool(((dw[0].double() - dot).abs() <= bound).all())
    del dy, out, row, w, dw, terms, dot, bound, on
    torch.cuda.empty_cache()


def test_dispatch_buffers_without_rows():
    """No row at all (every token absent): zeros for dx and the weights' gradient."""
    say("case: row gradients, no dispatch rows")
    R, T, K, H = 2, 30, 4, 64
    none = to_dev(np.full((R, T, K), -1))
    rows = torch.empty(0, H, dtype=torch.bfloat16, device=DEV)
    tok = torch.full((R, T, H), 77, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    w = torch.ones(R, T, K, device=DEV)
    assert (bits(U.permute_grad(rows, none, tok.clone())) == 0).all()
    assert (bits(U.combine(rows, none, w, tok.clone())) == 0).all()
    dw = torch.full((R, T, K), 9.0, device=DEV)
    dout, got = U.combine_grad(tok, rows, none, w, torch.empty_like(rows), dw)
    assert got is dw and dout.shape == (0, H) and (host(dw) == 0).all()
    U.combine_grad(tok, rows, none, w, rows, dw)
    assert U.combine_grad(tok, None, none, w, rows)[1] is None
    bad = none.clone()
    bad[1, 3, 2] = 0
    for call in (lambda e: U.permute_grad(rows, bad, tok.clone(), err=e),
                 lambda e: U.combine(rows, bad, w, tok.clone(), err=e),
                 lambda e: U.combine_grad(tok, rows, bad, w, rows, dw, err=e)):
        err = err_word()
        call(err)
        assert int(host(err)[0]) == U.ERR_ROW_RANGE
    assert (host(dw) == 0).all()


# More tokens than the calls spread over waves, slots in pairs, fours and eights, and rows of 1,
# 2, 4 and 8 vectors a lane, whole and ragged, up to more than one slice of 8 KiB.
@pytest.mark.parametrize("K", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("H", [64, 256, 512, 520, 1024, 1032, 2048, 7168])
def test_row_calls_of_many_tokens(K, H):
    say("case: row calls, many tokens", K, H)
    test_combine_grad((300 + K, 2, 520, K, 12, H, 0.1))
    test_permute_grad((400 + K, 2, 520, K, 12, H, 0.1))
    dr, dy, out, w = make(500 + K, 2, 520, K, 12, H, 0.1)
    for toks in (520, 30):                               # many tokens, and few
        d, wt = np.ascontiguousarray(dr[:, :toks]), np.ascontiguousarray(w[:, :toks])
        y = torch.full((2, toks, H), 77, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        U.combine(out, to_dev(d), to_dev(wt, torch.float32), y)
        assert np.array_equal(bits(y), O.combine(bits(out), d, wt))


@pytest.mark.parametrize("R,T,K,H", [
    (1, 13000, 8, 256),       # eight 512 B rows together
    (2, 9000, 5, 1024),       # four 2 KiB rows together
    (1, 20000, 3, 512),
    (1, 9000, 3, 1032),
])
def test_combine_grad_of_short_rows_in_phases(R, T, K, H):
    test_combine_grad_in_phases(R, T, K, H)
