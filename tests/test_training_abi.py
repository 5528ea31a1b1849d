"""Host-side refusals of the training calls (gate, row gradients, AdamW): they answer without
a GPU and before anything is enqueued."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_amd", "libuep.so")
OK, EINVAL, EGEOM, EWORKSPACE = 0, 1, 2, 3

i32, i64, f32, f64, sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                          ctypes.c_size_t)
null, fake, odd = ctypes.c_void_p(None), ctypes.c_void_p(4096), ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libuep.so is not built (run __graft_entry__.build())")
    return ctypes.CDLL(LIB)


def gate(lib, logits=fake, dtype=0, bias=null, R=2, T=3, E=8, K=2, score=0, scale=1.0, ids=fake,
         w=fake):
    return lib.uep_gate(logits, i32(dtype), bias, null, i32(R), i32(T), i32(E), i32(K), i32(score),
                        i32(1), f32(scale), ids, w, null, null)


def gate_grad(lib, dw=fake, logits=fake, dtype=0, R=2, T=3, E=8, K=2, score=0, scale=1.0, dl=fake):
    return lib.uep_gate_grad(dw, logits, i32(dtype), fake, fake, i32(R), i32(T), i32(E), i32(K),
                             i32(score), i32(1), f32(scale), dl, null, null)


@pytest.mark.parametrize("call", [gate, gate_grad])
def test_gate_refusals(lib, call):
    assert call(lib, T=0) == OK                                   # nothing to do
    for bad in (dict(R=0), dict(T=-1), dict(E=0), dict(K=0), dict(dtype=2), dict(dtype=-1),
                dict(score=2), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(logits=null)):
        assert call(lib, **bad) == EINVAL, bad
    for bad in (dict(R=65), dict(E=4097), dict(E=80, K=65), dict(K=9), dict(T=1 << 30),
                dict(T=1 << 25, K=1)):
        assert call(lib, **bad) == EGEOM, bad


def test_gate_pointers_and_bias(lib):
    assert gate(lib, ids=null) == EINVAL and gate(lib, w=null) == EINVAL
    assert gate(lib, bias=fake) == EINVAL                         # softmax takes no bias
    assert gate_grad(lib, dw=null) == EINVAL and gate_grad(lib, dl=null) == EINVAL


def permute_grad(lib, dout=fake, P=16, drow=fake, R=2, T=4, K=2, H=16, a=0, b=2, dx=fake):
    return lib.uep_permute_grad(dout, i64(P), drow, i32(R), i32(T), i32(K), i32(H), i32(a), i32(b),
                                dx, null, null)


def combine_grad(lib, dy=fake, out=fake, P=16, drow=fake, w=fake, R=2, T=4, K=2, H=16, a=0, b=2,
                 dout=fake, dw=fake):
    return lib.uep_combine_grad(dy, out, i64(P), drow, w, i32(R), i32(T), i32(K), i32(H), i32(a),
                                i32(b), dout, dw, null, null)


@pytest.mark.parametrize("call", [permute_grad, combine_grad])
def test_row_gradient_refusals(lib, call):
    assert call(lib, a=1, b=1) == OK and call(lib, T=0) == OK
    for bad in (dict(R=0), dict(T=-1), dict(K=0), dict(H=0), dict(P=-1), dict(a=-1), dict(b=3),
                dict(a=2, b=1), dict(dout=null), dict(drow=null)):
        assert call(lib, **bad) == EINVAL, bad
    for bad in (dict(H=12), dict(K=65), dict(T=1 << 30), dict(H=(1 << 29) + 8), dict(dout=odd)):
        assert call(lib, **bad) == EGEOM, bad


def test_row_gradient_pointers(lib):
    assert permute_grad(lib, dx=null) == EINVAL and permute_grad(lib, dx=odd) == EGEOM
    for bad in (dict(dy=null), dict(w=null), dict(out=null), dict(dw=null)):
        assert combine_grad(lib, **bad) == EINVAL, bad            # out and dw go together
    assert combine_grad(lib, dy=odd) == EGEOM and combine_grad(lib, out=odd) == EGEOM


def test_overlapping_buffers_are_refused(lib):
    """Outputs may not share bytes with inputs, except dout being `out` itself."""
    at = ctypes.c_void_p
    far = at(1 << 20)
    assert gate_grad(lib, logits=at(4096), dl=at(4096)) == EINVAL
    assert gate_grad(lib, logits=at(4096), dl=at(4096 + 2 * 3 * 8 * 4 - 4)) == EINVAL
    # R T H = 2 * 4 * 16 bf16 = 256 bytes, P H = 16 * 16 bf16 = 512 bytes
    assert permute_grad(lib, dout=at(4096), dx=at(4096 + 496)) == EINVAL
    assert permute_grad(lib, dout=at(4096 + 240), dx=at(4096)) == EINVAL
    assert combine_grad(lib, dy=at(4096), dout=at(4096 + 240), out=far) == EINVAL
    assert combine_grad(lib, dy=far, dout=at(4096), out=at(4096 + 496)) == EINVAL


class Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "tops", "copy")] + \
        [("n", i64), ("wd", f32), ("lr", f32)]


def table(**kw):
    d = dict(param=4096, grad=8192, m=12288, v=16384, tops=None, copy=None, n=10, wd=0.0, lr=1.0)
    d.update(kw)
    return (Tensor * 1)(Tensor(**d))


def prepare(lib, t, count=1, pd=0, gd=0, bits=32, plan=fake, size=1 << 20, tiles=True):
    n = i64(-1)
    return lib.uep_adamw_prepare(t, i32(count), i32(pd), i32(gd), i32(bits), plan, sz(size),
                                 ctypes.byref(n) if tiles else null, null)


def test_adamw_prepare_refusals(lib):
    lib.uep_adamw_plan_size.restype = sz
    one = lib.uep_adamw_plan_size(table(), i32(1))
    assert 0 < one < lib.uep_adamw_plan_size(table(n=1 << 20), i32(1))
    assert lib.uep_adamw_plan_size(table(n=-1), i32(1)) == 0
    assert prepare(lib, table(), size=one - 1) == EWORKSPACE
    for bad in (dict(count=-1), dict(pd=2), dict(gd=-1), dict(bits=16), dict(plan=null),
                dict(tiles=False)):
        assert prepare(lib, table(), **bad) == EINVAL, bad
    assert prepare(lib, null, count=1) == EINVAL
    for bad in (dict(n=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None),
                dict(wd=float("nan")), dict(lr=float("inf"))):
        assert prepare(lib, table(**bad)) == EINVAL, bad
    assert prepare(lib, table(), bits=8) == EINVAL                # 8-bit states need tops
    assert prepare(lib, table(copy=4096), pd=1) == EINVAL         # a copy of bf16 parameters
    for bad in (dict(n=(1 << 33) + 1), dict(param=4098), dict(m=12289), dict(copy=4097)):
        assert prepare(lib, table(**bad)) == EGEOM, bad
    assert prepare(lib, table(), plan=ctypes.c_void_p(4100)) == EGEOM
    assert prepare(lib, table(), count=65536) == EGEOM


def adamw(lib, plan=fake, tiles=1, pd=0, gd=0, bits=32, step=fake, sched=fake, b1=0.9, b2=0.999,
          eps=1e-8):
    return lib.uep_adamw(plan, i64(tiles), i32(pd), i32(gd), i32(bits), step, sched, f64(b1),
                         f64(b2), f64(eps), ctypes.c_uint32(0), null, null)


def test_adamw_refusals(lib):
    assert adamw(lib, tiles=0, plan=null) == OK
    nan = float("nan")
    for bad in (dict(tiles=-1), dict(pd=3), dict(gd=2), dict(bits=4), dict(plan=null),
                dict(step=null), dict(sched=null), dict(b1=1.0), dict(b1=-0.1), dict(b2=nan),
                dict(eps=0.0), dict(eps=nan), dict(eps=float("inf"))):
        assert adamw(lib, **bad) == EINVAL, bad
    assert adamw(lib, tiles=1 << 24) == EGEOM


def decode(lib, mc=fake, vc=fake, tops=fake, n=10, dtype=0, m=fake, v=fake):
    return lib.uep_adamw_decode(mc, vc, tops, i64(n), i32(dtype), m, v, null)


def test_adamw_decode_refusals(lib):
    assert decode(lib, n=0, mc=null) == OK
    for bad in (dict(n=-1), dict(dtype=2), dict(mc=null), dict(vc=null), dict(tops=null),
                dict(m=null), dict(v=null)):
        assert decode(lib, **bad) == EINVAL, bad


def test_binding_refuses_what_the_kernels_would_misread(lib):
    import torch
    from moe_expert_load_amd import uep as U
    x = torch.zeros(2, 3, 8)
    ids = torch.zeros(2, 3, 2, dtype=torch.int32)
    w = torch.zeros(2, 3, 2)
    for call, match in (
            (lambda: U.gate(x[0], 2), "R"),
            (lambda: U.gate(x.half(), 2), "float32 or bfloat16"),
            (lambda: U.gate(x, 2, bias=torch.zeros(7), score=1), "bias"),
            (lambda: U.gate(x, 2, topk_ids=ids[:, :, :1].contiguous()), "topk_ids"),
            (lambda: U.gate(x, 2, topk_ids=ids, gate_w=w.double()), "gate_w"),
            (lambda: U.gate(x, 2, batch_size=torch.zeros(1, dtype=torch.int32)), "batch_size"),
            (lambda: U.gate_grad(w[:1], x, ids, w), "dgate_w"),
            (lambda: U.gate_grad(w, x, ids.long(), w), "topk_ids"),
            (lambda: U.gate_grad(w, x, ids, w, dlogits=x.bfloat16()), "dlogits"),
            (lambda: U.gate(x, 2, topk_ids=ids, gate_w=w), "device memory")):
        with pytest.raises(TypeError, match=match):
            call()
    b = torch.bfloat16
    rows, tok = torch.zeros(9, 16, dtype=b), torch.zeros(2, 3, 16, dtype=b)
    for call, match in (
            (lambda: U.permute_grad(rows.float(), ids, tok), "dout"),
            (lambda: U.permute_grad(rows, ids, tok[:1]), "dx"),
            (lambda: U.permute_grad(rows[0], ids, tok), "dout"),
            (lambda: U.combine_grad(tok[:, :2], rows, ids, w, rows), "dy"),
            (lambda: U.combine_grad(tok, rows[:8], ids, w, rows), "out"),
            (lambda: U.combine_grad(tok, rows, ids, w[:1], rows), "gate_w"),
            (lambda: U.combine_grad(tok, rows, ids, w, rows, w[:1]), "dgate_w"),
            (lambda: U.combine_grad(tok, None, ids, w, rows, w), "needs the expert outputs"),
            (lambda: U.combine_grad(tok, rows, ids, w, rows, w), "device memory")):
        with pytest.raises(TypeError, match=match):
            call()


def test_adamw_binding_checks_its_lists(lib):
    import torch
    from moe_expert_load_amd import uep as U
    p, g, m, v = (torch.zeros(600) for _ in range(4))
    m8, v8 = m.to(torch.uint8), v.to(torch.uint8)
    tops = torch.zeros(3, dtype=torch.int32)
    for args, kw, match in (
            (([p], [g, g], [m], [v]), {}, "grads"),
            (([p], [g], [m], None), {}, "needed"),
            (([p.half()], [g], [m], [v]), {}, "float32 or bfloat16"),
            (([p], [g[:599]], [m], [v]), {}, "grads"),
            (([p], [g], [m8], [v8]), {}, "m\\[0\\]"),
            (([p], [g], [m], [v]), {"tops": [tops]}, "m\\[0\\]"),
            (([p.bfloat16()], [g], [m], [v]), {"copies": [p.bfloat16()]}, "copies"),
            (([p, p], [g, g], [m, m.clone()], [v, v.clone()]), {"weight_decay": [0.0]}, "weight"),
            (([p], [g], [m], [v]), {}, "device memory")):
        with pytest.raises(TypeError, match=match):
            U.adamw_prepare(*args, **kw)
    with pytest.raises(TypeError, match="AdamWPlan"):
        U.adamw(p, tops, m)
    with pytest.raises(TypeError, match="tops"):
        U.adamw_decode(m8, v8, tops[:2])


def test_float16_rows_are_refused(lib):
    """The row calls that compute read bf16; float16 elements would be taken for others."""
    import torch
    from moe_expert_load_amd import uep as U
    ids = torch.zeros(2, 3, 2, dtype=torch.int32)
    w = torch.zeros(2, 3, 2)

    def tensors(dtype):
        return torch.zeros(9, 16, dtype=dtype), torch.zeros(2, 3, 16, dtype=dtype)

    for dtype in (torch.bfloat16, torch.int16, torch.uint16):       # up to the device check
        rows, tok = tensors(dtype)
        for call in (lambda: U.permute_grad(rows, ids, tok), lambda: U.combine(rows, ids, w, tok),
                     lambda: U.combine_grad(tok, rows, ids, w, rows)):
            with pytest.raises(TypeError, match="device memory"):
                call()
    b_rows, b_tok = tensors(torch.bfloat16)
    for dtype in (torch.float16, torch.float32):
        rows, tok = tensors(dtype)
        for call, name in ((lambda: U.permute_grad(rows, ids, b_tok), "dout"),
                           (lambda: U.permute_grad(b_rows, ids, tok), "dx"),
                           (lambda: U.combine(rows, ids, w, b_tok), "out"),
                           (lambda: U.combine(b_rows, ids, w, tok), "y"),
                           (lambda: U.combine_grad(tok, b_rows, ids, w, b_rows), "dy"),
                           (lambda: U.combine_grad(b_tok, rows, ids, w, b_rows), "out"),
                           (lambda: U.combine_grad(b_tok, b_rows, ids, w, rows), "dout")):
            with pytest.raises(TypeError, match=name + " must hold"):
                call()


def test_outputs_may_not_share_memory_with_any_other_array(lib):
    """Every output against every other array of its call; 2 * 3 * 2 int32 or fp32 slots are 48
    bytes, 2 * 4 * 2 of the row calls 64."""
    at = ctypes.c_void_p
    base = 1 << 20

    def refused(call, args, out, allowed=()):
        for other in args:
            if other == out or other in allowed:
                continue
            for off in (0, args[other] - 4, 4 - args[out]):
                ptrs = {a: at(base * (i + 1)) for i, a in enumerate(args)}
                ptrs[out] = at(ptrs[other].value + off)
                assert call(ptrs) == EINVAL, (out, other, off)

    def call_gate(p):
        return lib.uep_gate(p["logits"], i32(0), p["bias"], p["bs"], i32(2), i32(3), i32(8), i32(2),
                            i32(1), i32(1), f32(1.0), p["ids"], p["w"], null, null)

    args = dict(logits=192, bias=32, bs=8, ids=48, w=48)
    refused(call_gate, args, "ids")
    refused(call_gate, args, "w")

    def call_gate_grad(p):
        return lib.uep_gate_grad(p["dw"], p["logits"], i32(0), p["ids"], p["w"], i32(2), i32(3),
                                 i32(8), i32(2), i32(1), i32(1), f32(1.0), p["dl"], null, null)

    refused(call_gate_grad, dict(dw=48, logits=192, ids=48, w=48, dl=192), "dl")

    def call_permute(p):
        return permute_grad(lib, dout=p["dout"], drow=p["drow"], dx=p["dx"])

    def call_combine(p):
        return combine_grad(lib, dy=p["dy"], out=p["out"], drow=p["drow"], w=p["w"],
                            dout=p["dout"], dw=p["dw"])

    # rows lie on 16 bytes: offsets of 4 are refused as geometry, so whole rows here
    for other, off in (("dout", 0), ("dout", 496), ("drow", 0), ("drow", 48)):
        p = {a: at(base * (i + 1)) for i, a in enumerate(("dout", "drow", "dx"))}
        p["dx"] = at(p[other].value + off)
        assert call_permute(p) == EINVAL, (other, off)
    names = ("dy", "out", "drow", "w", "dout", "dw")
    for other, off in (("dy", 0), ("dy", 240), ("drow", 0), ("drow", 48), ("w", 0), ("w", 48),
                       ("out", 496)):
        p = {a: at(base * (i + 1)) for i, a in enumerate(names)}
        p["dout"] = at(p[other].value + off)
        assert call_combine(p) == EINVAL, (other, off)
    refused(call_combine, dict(dy=256, out=512, drow=64, w=64, dout=512, dw=64), "dw")
