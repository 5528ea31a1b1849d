"""Host-side refusals of the balance loss, the rows in 8 bits and the experts' products: they
answer without a GPU and before anything is enqueued."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_amd", "libuep.so")
OK, EINVAL, EGEOM, EWORKSPACE = 0, 1, 2, 3

i32, i64, sz, at = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
null = at(None)


def mb(n):
    """Addresses far apart that nothing is read from."""
    return at(n << 24)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libuep.so is not built (run __graft_entry__.build())")
    lib = ctypes.CDLL(LIB)
    lib.uep_balance_loss_workspace_size.restype = sz
    return lib


def size(lib, R=2, T=6, E=8, G=2):
    return lib.uep_balance_loss_workspace_size(i32(R), i32(T), i32(E), i32(G))


def loss(lib, logits=mb(1), dtype=0, ids=mb(2), off=null, G=2, R=2, T=6, E=8, K=2, score=0,
         out=mb(3), counts=mb(4), prob=mb(5), tokens=mb(6), ws=mb(7), ws_bytes=1 << 20):
    return lib.uep_balance_loss(logits, i32(dtype), ids, off, i32(G), i32(R), i32(T), i32(E),
                                i32(K), i32(score), out, counts, prob, tokens, null, ws,
                                sz(ws_bytes), null)


def loss_grad(lib, logits=mb(1), dtype=0, ids=mb(2), off=null, G=2, R=2, T=6, E=8, K=2, score=0,
              dloss=mb(3), counts=mb(4), tokens=mb(6), add=null, dl=mb(7)):
    return lib.uep_balance_loss_grad(dloss, logits, i32(dtype), ids, counts, tokens, off, i32(G),
                                     i32(R), i32(T), i32(E), i32(K), i32(score), add, dl, null,
                                     null)


@pytest.mark.parametrize("call", [loss, loss_grad])
def test_balance_refusals(lib, call):
    for bad in (dict(R=0), dict(T=-1), dict(E=0), dict(K=0), dict(G=0), dict(dtype=2),
                dict(dtype=-1), dict(score=2), dict(logits=null), dict(ids=null),
                dict(counts=null), dict(tokens=null)):
        assert call(lib, **bad) == EINVAL, bad
    for bad in (dict(R=65), dict(E=4097), dict(K=65), dict(T=1 << 30), dict(T=1 << 25, K=1),
                dict(G=65536, off=mb(9)), dict(G=5), dict(T=1 << 24, R=1, K=1, G=3)):
        assert call(lib, **bad) == EGEOM, bad


def test_balance_pointers_and_workspace(lib):
    for bad in (dict(out=null), dict(prob=null)):
        assert loss(lib, **bad) == EINVAL
    need = size(lib)
    assert 0 < need < size(lib, T=1 << 20)
    assert size(lib, R=65) == size(lib, E=0) == size(lib, G=0) == size(lib, T=-1) == 0
    assert loss(lib, ws=null) == EWORKSPACE and loss(lib, ws_bytes=need - 1) == EWORKSPACE
    assert loss(lib, ws=at((7 << 24) + 4)) == EGEOM
    assert loss_grad(lib, T=0) == OK
    assert loss_grad(lib, dloss=null) == EINVAL and loss_grad(lib, dl=null) == EINVAL


def test_balance_overlaps(lib):
    """R T E = 96 fp32 = 384 bytes of logits, 2 * 8 counts = 64 bytes."""
    first = 1 << 24
    for bad in (dict(out=at(first + 380)), dict(counts=at(first - 60)), dict(prob=mb(4)),
                dict(tokens=at((4 << 24) + 60)), dict(ws=at(first + 368)), dict(out=mb(7))):
        assert loss(lib, **bad) == EINVAL, bad
    for bad in (dict(dl=at(first + 380)), dict(dl=mb(4)), dict(add=at((7 << 24) + 4)),
                dict(dl=mb(3)), dict(dl=mb(6)), dict(dl=mb(2))):
        assert loss_grad(lib, **bad) == EINVAL, bad


def rows(lib, x=mb(1), n=4, H=32, live=null, q=mb(2), s=mb(3)):
    return lib.uep_quant_rows(x, i64(n), i32(H), live, q, s, null, null)


def dispatch(lib, x=mb(1), row=mb(4), R=2, T=3, K=2, H=32, a=0, b=2, q=mb(2), s=mb(3), P=12):
    return lib.uep_permute_quant(x, row, i32(R), i32(T), i32(K), i32(H), i32(a), i32(b), q, s,
                                 i64(P), null, null)


def test_row_refusals(lib):
    assert rows(lib, n=0) == OK
    for bad in (dict(n=-1), dict(H=0), dict(x=null), dict(q=null), dict(s=null)):
        assert rows(lib, **bad) == EINVAL, bad
    for bad in (dict(H=24), dict(H=65552), dict(n=1 << 31), dict(x=at((1 << 24) + 8)),
                dict(q=at((2 << 24) + 8))):
        assert rows(lib, **bad) == EGEOM, bad
    for bad in (dict(q=at((1 << 24) + 240)), dict(s=at((1 << 24) + 252)), dict(s=mb(2)),
                dict(q=mb(5), live=at((5 << 24) + 124)), dict(s=mb(5), live=mb(5))):
        assert rows(lib, **bad) == EINVAL, bad


def test_dispatch_refusals(lib):
    assert dispatch(lib, T=0) == OK and dispatch(lib, a=1, b=1) == OK
    for bad in (dict(R=0), dict(T=-1), dict(K=0), dict(H=0), dict(P=-1), dict(a=-1), dict(b=3),
                dict(a=2, b=1), dict(x=null), dict(row=null), dict(q=null), dict(s=null)):
        assert dispatch(lib, **bad) == EINVAL, bad
    for bad in (dict(R=65), dict(K=65), dict(H=24), dict(H=65552), dict(T=1 << 30),
                dict(P=1 << 31), dict(x=at((1 << 24) + 8)), dict(q=at((2 << 24) + 8))):
        assert dispatch(lib, **bad) == EGEOM, bad
    for bad in (dict(q=at((1 << 24) + 368)), dict(q=mb(4)), dict(s=mb(4)), dict(s=mb(2)),
                dict(s=mb(1))):
        assert dispatch(lib, **bad) == EINVAL, bad


def product(lib, q=mb(1), s=mb(2), n=4, off=mb(3), R=2, E=4, S=1, w=mb(4), ws=mb(5), sw=mb(6),
            ss=mb(7), N=16, D=32, act=0, out=mb(8)):
    return lib.uep_expert_product(q, s, i64(n), off, i32(R), i32(E), i32(S), w, ws, sw, ss, i32(N),
                                  i32(D), i32(act), out, null, null)


def test_product_refusals(lib):
    assert product(lib, n=0) == OK
    for bad in (dict(n=-1), dict(R=0), dict(E=0), dict(S=-1), dict(N=0), dict(D=0), dict(act=2),
                dict(act=-1), dict(off=null), dict(q=null), dict(s=null), dict(w=null),
                dict(ws=null), dict(sw=null), dict(ss=null), dict(out=null)):
        assert product(lib, **bad) == EINVAL, bad
    for bad in (dict(R=65, E=65), dict(E=5), dict(E=4098), dict(S=9), dict(N=12), dict(D=24),
                dict(D=65552), dict(N=24, act=1), dict(N=1 << 16, D=1 << 15), dict(n=1 << 31),
                dict(n=(1 << 29) + 1), dict(q=at((1 << 24) + 8)), dict(w=at((4 << 24) + 8)), dict(sw=at((6 << 24) + 8)),
                dict(out=at((8 << 24) + 8))):
        assert product(lib, **bad) == EGEOM, bad
    one = dict(R=1, E=1, S=0, sw=null, ss=null)
    assert product(lib, off=null, n=0, **one) == OK
    # out: 4 rows of 16 bf16 = 128 bytes
    for bad in (dict(out=at((1 << 24) + 112)), dict(out=mb(2)), dict(out=mb(3)),
                dict(out=at((4 << 24) - 112)), dict(out=mb(5)), dict(out=mb(6)), dict(out=mb(7))):
        assert product(lib, **bad) == EINVAL, bad
