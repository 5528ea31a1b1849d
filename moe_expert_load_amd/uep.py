"""Thin Python binding of libuep.so (the C-ABI in include/uep.h).

Argument marshalling only: torch supplies device memory and the HIP stream; every
step of the balancing path runs in the library's HIP kernels.  Output tensors the
caller does not pass are allocated with torch on the input's device.  With `stream` a
call works on that stream, which the caller orders with the streams that make its inputs
and use its outputs (what the call allocates is safe by itself).  A non-zero status
raises UEPError.  Importing this module fails loudly when the library is
not built: there is no fallback path.
"""

from __future__ import annotations

import bisect
import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libuep.so")

OK, EINVAL, EGEOM, EWORKSPACE, EHIP = 0, 1, 2, 3, 4
ERR_ID_RANGE, ERR_DUP_ID, ERR_QUOTA_SUM, ERR_INST_DUP = 1, 2, 4, 8
ERR_BAD_QUOTA, ERR_COVER, ERR_LP, ERR_ROW_RANGE = 16, 32, 64, 128
ERR_LOGIT, ERR_GRAD, ERR_PLAN = 256, 512, 1024
STAGE_WEIGHTS, STAGE_GRAD_REDUCE = 0, 1
F32, BF16 = 0, 1
GATE_SOFTMAX, GATE_SIGMOID = 0, 1
ADAMW_BLOCK = 256       # elements of one tensor that share an entry of `tops` (8-bit states)

_P = ctypes.c_void_p
_I = ctypes.c_int32
_I64 = ctypes.c_int64
_U64 = ctypes.c_uint64
_SZ = ctypes.c_size_t
_U32 = ctypes.c_uint32
_F = ctypes.c_float
_D = ctypes.c_double

# name -> (restype, argtypes); the exact list of symbols include/uep.h declares
SIGNATURES = {
    "uep_version": (ctypes.c_char_p, []),
    "uep_status_string": (ctypes.c_char_p, [_I]),
    "uep_device_copy": (_I, [_P, _P, _I64, _P]),
    "uep_device_fill": (_I, [_P, _I64, ctypes.c_uint32, _P]),
    "uep_load_matrix_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "uep_load_matrix": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "uep_load_matrix_noalloc": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "uep_solve_quota": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "uep_identity_quota": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "uep_reroute_workspace_size": (_SZ, [_I, _I, _I]),
    "uep_reroute_assign": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _I,
                                _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "uep_plan_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "uep_plan": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                      _P, _P, _P, _SZ, _P]),
    "uep_permute": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _I64, _P, _P, _P]),
    "uep_combine": (_I, [_P, _I64, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "uep_stage_replica_weights": (_I, [_I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _I64, _P]),
    "uep_waterfill": (_I, [_P, _P, _P, _I, _I, _I, _I, _U64, _U64, _I, _I, _P, _P, _P, _P, _P,
                           _P]),
    "uep_lplb_struct_size": (_SZ, [_I, _I, _I]),
    "uep_lplb_prepare": (_I, [_P, _I, _I, _I, _P, _SZ, _P]),
    "uep_lplb_sample": (_I, [_P, _I, _I, _I, _P, _P, _U64, _U64, _P, _P, _P]),
    "uep_lplb": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P]),
    "uep_lplb_plan_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "uep_lplb_plan": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _I, _I, _I] + [_P] * 12 + [_SZ, _P]),
    "uep_gate": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P]),
    "uep_gate_grad": (_I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "uep_permute_grad": (_I, [_P, _I64, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "uep_combine_grad": (_I, [_P, _P, _I64, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "uep_adamw_plan_size": (_SZ, [_P, _I]),
    "uep_adamw_prepare": (_I, [_P, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "uep_adamw": (_I, [_P, _I64, _I, _I, _I, _P, _P, _D, _D, _D, _U32, _P, _P]),
    "uep_adamw_decode": (_I, [_P, _P, _P, _I64, _I, _P, _P, _P]),
}


class UEPError(RuntimeError):
    pass


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def version() -> str:
    return LIB.uep_version().decode()


def _check(status: int, name: str) -> None:
    if status != OK:
        raise UEPError(f"{name}: {LIB.uep_status_string(status).decode()} (status {status})")


def _p(t: Optional[torch.Tensor]):
    """Device pointer of a contiguous GPU tensor (None stays NULL).  A host tensor is
    refused here: its address handed to a kernel would fault the device."""
    if t is None:
        return None
    if not t.is_cuda:
        raise TypeError("the library takes device memory: got a tensor on " + str(t.device))
    if not t.is_contiguous():
        raise TypeError("the library takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object around it, which costs 3 us a call: a
# third of what a small call takes.
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream) -> ctypes.c_void_p:
    if stream is None:
        if _RAW_STREAM is not None:
            return ctypes.c_void_p(_RAW_STREAM(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _i32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor")
    return t


def _fresh(shape, dtype, device, stream) -> torch.Tensor:
    """Memory that a call allocates and writes on `stream`.  It is the current stream's, which
    may still have work queued for whoever held it last: another stream waits for that, and the
    memory is not given away again before that stream has passed the call."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None and t.is_cuda and stream.cuda_stream != (_s(None).value or 0):
        stream.wait_stream(torch.cuda.current_stream())
        t.record_stream(stream)
    return t


def _new(shape, like: torch.Tensor, stream, dtype=torch.int32) -> torch.Tensor:
    return _fresh(shape, dtype, like.device, stream)


def _table_stream(buf: torch.Tensor, home: int, stream) -> ctypes.c_void_p:
    """The stream of a call that reads `buf`, a table made while `home` was current: on any
    other, the table's memory is not given away before that stream has passed the call, so the
    table may be dropped while it runs."""
    s = _s(stream)
    if (s.value or 0) != home:
        buf.record_stream(torch.cuda.current_stream() if stream is None else stream)
    return s


def _buf(t: Optional[torch.Tensor], n: int, name: str, dtype=torch.int32):
    """A caller's buffer for the library to read or write: contiguous, of `dtype` (any
    16-bit type for torch.int16), with at least n elements, since the kernels index it
    by the geometry alone.  None stays None."""
    if t is None:
        return None
    ok_type = t.element_size() == 2 if dtype == torch.int16 else t.dtype == dtype
    if not ok_type or not t.is_contiguous() or t.numel() < n:
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of at least {n} elements")
    return t


# ---------------------------------------------------------------------------
def load_matrix_workspace_size(R, T, K, E) -> int:
    return int(LIB.uep_load_matrix_workspace_size(R, T, K, E))


def load_matrix(topk_ids, E, counts=None, bucket_pos=None, err=None, ws=None, stream=None,
                counts_only=False):
    """counts [R][E] and bucket_pos [R][T][K]; with counts_only=True the positions are
    not computed and None is returned in their place."""
    _i32(topk_ids, "topk_ids")
    R, T, K = topk_ids.shape
    counts = _new((R, E), topk_ids, stream) if counts is None else _buf(counts, R * E, "counts")
    if counts_only:
        bucket_pos = None
    elif bucket_pos is None:
        bucket_pos = _new((R, T, K), topk_ids, stream)
    else:
        _buf(bucket_pos, R * T * K, "bucket_pos")
    _buf(err, 1, "err")
    n = load_matrix_workspace_size(R, T, K, E)
    ws = _new((max(n, 4),), topk_ids, stream, torch.uint8) if ws is None else ws
    _check(LIB.uep_load_matrix(_p(topk_ids), R, T, K, E, _p(counts), _p(bucket_pos), _p(err),
                               _p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "uep_load_matrix")
    return counts, bucket_pos


def load_matrix_noalloc(topk_ids, E, counts=None, bucket_pos=None, err=None, stream=None,
                        counts_only=False):
    """uep_load_matrix_noalloc: as load_matrix, with the library's own per-device scratch
    instead of a workspace (pass counts / bucket_pos to allocate nothing here either)."""
    _i32(topk_ids, "topk_ids")
    R, T, K = topk_ids.shape
    counts = _new((R, E), topk_ids, stream) if counts is None else _buf(counts, R * E, "counts")
    if counts_only:
        bucket_pos = None
    elif bucket_pos is None:
        bucket_pos = _new((R, T, K), topk_ids, stream)
    else:
        _buf(bucket_pos, R * T * K, "bucket_pos")
    _buf(err, 1, "err")
    _check(LIB.uep_load_matrix_noalloc(_p(topk_ids), R, T, K, E, _p(counts), _p(bucket_pos),
                                       _p(err), _s(stream)), "uep_load_matrix_noalloc")
    return counts, bucket_pos


def solve_quota(counts, S, q_min, out=None, stream=None):
    _i32(counts, "counts")
    R, E = counts.shape
    ipr = E // R + S
    o = out or {}
    slot_expert, inst_expert, inst_quota, rank_load, stats = (
        o[name] if name in o else _new(shape, counts, stream)
        for name, shape in (("slot_expert", (R, max(S, 1))), ("inst_expert", (R * ipr,)),
                            ("inst_quota", (R * ipr,)), ("rank_load", (R,)), ("stats", (4,))))
    for name, t, n in (("slot_expert", slot_expert, R * S), ("inst_expert", inst_expert, R * ipr),
                       ("inst_quota", inst_quota, R * ipr), ("rank_load", rank_load, R),
                       ("stats", stats, 4)):
        _buf(t, n, name)
    _check(LIB.uep_solve_quota(_p(counts), R, E, S, q_min, _p(slot_expert), _p(inst_expert),
                               _p(inst_quota), _p(rank_load), _p(stats), _s(stream)),
           "uep_solve_quota")
    return {"slot_expert": slot_expert[:, :S], "inst_expert": inst_expert,
            "inst_quota": inst_quota, "rank_load": rank_load, "stats": stats,
            "inst_per_rank": ipr}


def identity_quota(counts, inst_expert, inst_quota=None, stream=None):
    _i32(counts, "counts")
    R, E = counts.shape
    _i32(inst_expert, "inst_expert")
    n = inst_expert.numel()
    inst_quota = _new((n,), counts, stream) if inst_quota is None \
        else _buf(inst_quota, n, "inst_quota")
    _check(LIB.uep_identity_quota(_p(counts), R, E, n, _p(inst_expert), _p(inst_quota),
                                  _s(stream)), "uep_identity_quota")
    return inst_quota


def reroute_workspace_size(R, E, inst_per_rank) -> int:
    return int(LIB.uep_reroute_workspace_size(R, E, inst_per_rank))


def reroute_assign(counts, topk_ids, bucket_pos, inst_per_rank, inst_expert, inst_quota,
                   r_begin=0, r_end=None, xfer=None, inst_offset=None, dest_inst=None,
                   dest_row=None, err=None, ws=None, stream=None):
    _i32(counts, "counts")
    _i32(topk_ids, "topk_ids")
    R, E = counts.shape
    _, T, K = topk_ids.shape
    r_end = R if r_end is None else r_end
    I = R * inst_per_rank
    _buf(bucket_pos, R * T * K, "bucket_pos")
    _buf(inst_expert, I, "inst_expert")
    _buf(inst_quota, I, "inst_quota")
    _buf(err, 1, "err")
    xfer = _new((R, I), counts, stream) if xfer is None else _buf(xfer, R * I, "xfer")
    inst_offset = _new((I + 1,), counts, stream) if inst_offset is None \
        else _buf(inst_offset, I + 1, "inst_offset")
    dest_inst = _new((R, T, K), counts, stream) if dest_inst is None \
        else _buf(dest_inst, R * T * K, "dest_inst")
    dest_row = _new((R, T, K), counts, stream) if dest_row is None \
        else _buf(dest_row, R * T * K, "dest_row")
    n = reroute_workspace_size(R, E, inst_per_rank)
    ws = _new((max(n, 4),), counts, stream, torch.uint8) if ws is None else ws
    _check(LIB.uep_reroute_assign(_p(counts), _p(topk_ids), _p(bucket_pos), R, T, K, E,
                                  inst_per_rank, _p(inst_expert), _p(inst_quota), r_begin, r_end,
                                  _p(xfer), _p(inst_offset), _p(dest_inst), _p(dest_row),
                                  _p(err), _p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "uep_reroute_assign")
    return xfer, inst_offset, dest_inst, dest_row


def plan_workspace_size(R, T, K, E, S) -> int:
    return int(LIB.uep_plan_workspace_size(R, T, K, E, S))


def plan(topk_ids, E, S, q_min, r_begin=0, r_end=None, out=None, err=None, ws=None, stream=None):
    """uep_plan: load matrix, quota solve and reroute/assignment in one call.  `out` may
    hold preallocated buffers under the keys below; returns that dict."""
    _i32(topk_ids, "topk_ids")
    R, T, K = topk_ids.shape
    r_end = R if r_end is None else r_end
    ipr = E // R + S
    I = R * ipr
    shapes = {"counts": (R, E), "bucket_pos": (R, T, K), "slot_expert": (R, max(S, 1)),
              "inst_expert": (I,), "inst_quota": (I,), "rank_load": (R,), "stats": (4,),
              "xfer": (R, I), "inst_offset": (I + 1,), "dest_inst": (R, T, K),
              "dest_row": (R, T, K)}
    o = {} if out is None else dict(out)
    for k, shp in shapes.items():
        n = 1
        for d in shp:
            n *= d
        o[k] = _new(shp, topk_ids, stream) if o.get(k) is None else _buf(o[k], n, k)
    _buf(err, 1, "err")
    need = plan_workspace_size(R, T, K, E, S)
    ws = _new((max(need, 4),), topk_ids, stream, torch.uint8) if ws is None else ws
    _check(LIB.uep_plan(_p(topk_ids), R, T, K, E, S, q_min, r_begin, r_end, _p(o["counts"]),
                        _p(o["bucket_pos"]), _p(o["slot_expert"]), _p(o["inst_expert"]),
                        _p(o["inst_quota"]), _p(o["rank_load"]), _p(o["stats"]), _p(o["xfer"]),
                        _p(o["inst_offset"]), _p(o["dest_inst"]), _p(o["dest_row"]), _p(err),
                        _p(ws), ws.numel() * ws.element_size(), _s(stream)), "uep_plan")
    o["inst_per_rank"] = ipr
    return o


def permute(x, dest_row, out, row_src=None, r_begin=0, r_end=None, stream=None, err=None):
    """x [R][T][H] bf16 (or 16-bit) tensor; out [P][H] of the same dtype (P rows bound
    the dispatch rows: an entry of dest_row outside [-1, P) is skipped and flagged)."""
    R, T, H = x.shape
    _i32(dest_row, "dest_row")
    K = dest_row.shape[2]
    r_end = R if r_end is None else r_end
    if x.element_size() != 2 or out.element_size() != 2:
        raise TypeError("x and out must hold 16-bit elements")
    if tuple(dest_row.shape) != (R, T, K) or out.dim() != 2 or out.shape[1] != H:
        raise TypeError("dest_row must be [R][T][K] and out [P][H] for x [R][T][H]")
    if row_src is not None:
        _i32(row_src, "row_src")
        if row_src.numel() != out.shape[0]:
            raise TypeError("row_src must have one entry per row of out")
    _check(LIB.uep_permute(_p(x), _p(dest_row), R, T, K, H, r_begin, r_end, _p(out), out.shape[0],
                           _p(row_src), _p(err), _s(stream)), "uep_permute")
    return out, row_src


def _bf16_rows(t: torch.Tensor, shape, name: str) -> None:
    """bf16 rows that a call computes with, of exactly this shape (the kernels index them by
    the geometry): bfloat16, or their bits in 16-bit integers.  float16 would be misread."""
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name} must hold 16-bit elements, bfloat16 or its bits as int16 or "
                        f"uint16, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise TypeError(f"{name} must be of shape {list(shape)}, got {list(t.shape)}")


def combine(out, dest_row, gate_w, y, r_begin=0, r_end=None, stream=None, err=None):
    """out [P][H] bf16 dispatch buffer; dest_row [R][T][K] int32; gate_w [R][T][K]
    float32; y [R][T][H] bf16 (rows of ranks in [r_begin, r_end) are written)."""
    _i32(dest_row, "dest_row")
    if out.dim() != 2 or dest_row.dim() != 3:
        raise TypeError("out must be [P][H] and dest_row [R][T][K]")
    R, T, K = dest_row.shape
    H = out.shape[1]
    r_end = R if r_end is None else r_end
    _bf16_rows(out, (out.shape[0], H), "out")
    if gate_w.dtype != torch.float32 or tuple(gate_w.shape) != (R, T, K):
        raise TypeError("gate_w must be float32 [R][T][K]")
    _bf16_rows(y, (R, T, H), "y")
    _check(LIB.uep_combine(_p(out), out.shape[0], _p(dest_row), _p(gate_w), R, T, K, H, r_begin,
                           r_end, _p(y), _p(err), _s(stream)), "uep_combine")
    return y


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def gate(logits, K, bias=None, batch_size=None, score=GATE_SOFTMAX, renorm=True, scale=1.0,
         topk_ids=None, gate_w=None, err=None, stream=None):
    """Router gate: logits [R][T][E] float32 or bfloat16 -> topk_ids [R][T][K] int32 (ties to
    the lowest id, -1 where no expert is eligible) and gate_w [R][T][K] float32."""
    if logits.dim() != 3:
        raise TypeError("logits must be [R][T][E]")
    R, T, E = logits.shape
    dt = _dtype(logits, "logits")
    _buf(bias, E, "bias", torch.float32)
    _buf(batch_size, R, "batch_size")
    _buf(err, 1, "err")
    n = R * T * K
    topk_ids = _new((R, T, K), logits, stream) if topk_ids is None \
        else _buf(topk_ids, n, "topk_ids")
    gate_w = _new((R, T, K), logits, stream, torch.float32) if gate_w is None \
        else _buf(gate_w, n, "gate_w", torch.float32)
    _check(LIB.uep_gate(_p(logits), dt, _p(bias), _p(batch_size), R, T, E, K, score,
                        1 if renorm else 0, scale, _p(topk_ids), _p(gate_w), _p(err), _s(stream)),
           "uep_gate")
    return topk_ids, gate_w


def gate_grad(dgate_w, logits, topk_ids, gate_w, score=GATE_SOFTMAX, renorm=True, scale=1.0,
              dlogits=None, err=None, stream=None):
    """Gradient of gate's weights: dgate_w [R][T][K] float32 -> dlogits [R][T][E] of the
    logits' dtype, given what gate took and wrote."""
    if logits.dim() != 3 or topk_ids.dim() != 3:
        raise TypeError("logits must be [R][T][E] and topk_ids [R][T][K]")
    R, T, E = logits.shape
    dt = _dtype(logits, "logits")
    _i32(topk_ids, "topk_ids")
    if tuple(topk_ids.shape[:2]) != (R, T):
        raise TypeError("logits and topk_ids must have the same [R][T]")
    K = topk_ids.shape[2]
    _buf(gate_w, R * T * K, "gate_w", torch.float32)
    _buf(dgate_w, R * T * K, "dgate_w", torch.float32)
    _buf(err, 1, "err")
    dlogits = _new((R, T, E), logits, stream, logits.dtype) if dlogits is None \
        else _buf(dlogits, R * T * E, "dlogits", logits.dtype)
    if dlogits.dtype != logits.dtype:
        raise TypeError("dlogits must have the logits' dtype")
    _check(LIB.uep_gate_grad(_p(dgate_w), _p(logits), dt, _p(topk_ids), _p(gate_w), R, T, E, K,
                             score, 1 if renorm else 0, scale, _p(dlogits), _p(err), _s(stream)),
           "uep_gate_grad")
    return dlogits


def permute_grad(dout, dest_row, dx, r_begin=0, r_end=None, stream=None, err=None):
    """Gradient of permute: dout [P][H] bf16 -> dx [R][T][H] bf16, the sum over every token's
    dispatch rows (rows of ranks in [r_begin, r_end) are written)."""
    _i32(dest_row, "dest_row")
    if dout.dim() != 2 or dest_row.dim() != 3:
        raise TypeError("dout must be [P][H] and dest_row [R][T][K]")
    R, T, K = dest_row.shape
    P, H = dout.shape
    r_end = R if r_end is None else r_end
    _bf16_rows(dout, (P, H), "dout")
    _bf16_rows(dx, (R, T, H), "dx")
    _buf(err, 1, "err")
    _check(LIB.uep_permute_grad(_p(dout), P, _p(dest_row), R, T, K, H, r_begin, r_end, _p(dx),
                                _p(err), _s(stream)), "uep_permute_grad")
    return dx


def combine_grad(dy, out, dest_row, gate_w, dout, dgate_w=None, r_begin=0, r_end=None,
                 stream=None, err=None):
    """Gradients of combine: dy [R][T][H] bf16 -> dout [P][H] bf16 (the gradient of the expert
    outputs; may be `out` itself) and dgate_w [R][T][K] float32.  With out None only dout is
    computed."""
    _i32(dest_row, "dest_row")
    if dout.dim() != 2 or dest_row.dim() != 3:
        raise TypeError("dout must be [P][H] and dest_row [R][T][K]")
    R, T, K = dest_row.shape
    P, H = dout.shape
    r_end = R if r_end is None else r_end
    _bf16_rows(dy, (R, T, H), "dy")
    _bf16_rows(dout, (P, H), "dout")
    if gate_w.dtype != torch.float32 or tuple(gate_w.shape) != (R, T, K):
        raise TypeError("gate_w must be float32 [R][T][K]")
    if out is None:
        if dgate_w is not None:
            raise TypeError("dgate_w needs the expert outputs `out`")
    else:
        _bf16_rows(out, (P, H), "out")
        dgate_w = _new((R, T, K), dy, stream, torch.float32) if dgate_w is None else dgate_w
        if dgate_w.dtype != torch.float32 or tuple(dgate_w.shape) != (R, T, K):
            raise TypeError("dgate_w must be float32 [R][T][K]")
    _buf(err, 1, "err")
    _check(LIB.uep_combine_grad(_p(dy), _p(out), P, _p(dest_row), _p(gate_w), R, T, K, H, r_begin,
                                r_end, _p(dout), _p(dgate_w), _p(err), _s(stream)),
           "uep_combine_grad")
    return dout, dgate_w


class AdamWTensor(ctypes.Structure):
    """struct uep_adamw_tensor of include/uep.h."""

    _fields_ = [("param", _P), ("grad", _P), ("m", _P), ("v", _P), ("tops", _P), ("copy", _P),
                ("n", _I64), ("weight_decay", _F), ("lr_scale", _F)]


@dataclasses.dataclass(frozen=True)
class AdamWPlan:
    """A table of tensors from adamw_prepare: the device buffer, the sizes and types every
    step passes back, the tensors themselves, which the plan points into, and the stream that
    was current (`home`).  It may be dropped while a step runs; tensors that are dropped with it
    have to be recorded on the step's stream like any others."""

    buf: torch.Tensor
    n_tiles: int
    param_dtype: int
    grad_dtype: int
    state_bits: int
    tensors: tuple
    home: int = 0


def _per_tensor(x, n, name):
    x = [float(x)] * n if isinstance(x, (int, float)) else [float(v) for v in x]
    if len(x) != n:
        raise TypeError(f"{name} must be one number or one for each of the {n} tensors")
    return x


def adamw_prepare(params, grads, m, v, copies=None, tops=None, weight_decay=0.0, lr_scale=1.0,
                  device=None, stream=None) -> AdamWPlan:
    """Offline: the plan of an AdamW step over lists of contiguous tensors.  params and grads
    float32 or bfloat16 (one type each); m and v float32, or uint8 with `tops` (int32, one entry
    per 256 elements) for 8-bit states; copies (bfloat16, optional) take the new values of
    float32 params.  weight_decay and lr_scale: one number, or one per tensor."""
    n = len(params)
    lists = {"grads": grads, "m": m, "v": v, "copies": copies, "tops": tops}
    for name, x in lists.items():
        if x is not None and len(x) != n:
            raise TypeError(f"{name} must have one tensor for each of the {n} params")
    if m is None or v is None or grads is None:
        raise TypeError("grads, m and v are needed")
    bits = 8 if tops is not None else 32
    state = torch.uint8 if bits == 8 else torch.float32
    pd = _dtype(params[0], "params") if n else F32
    gd = _dtype(grads[0], "grads") if n else F32
    if copies is not None and pd != F32:
        raise TypeError("copies go with float32 params")
    wd, ls = _per_tensor(weight_decay, n, "weight_decay"), _per_tensor(lr_scale, n, "lr_scale")
    sizes = [p.numel() for p in params]
    dev = params[0].device if n else torch.device("cuda" if device is None else device)
    lists = [("params", params, params[0].dtype if n else None, sizes),
             ("grads", grads, grads[0].dtype if n else None, sizes), ("m", m, state, sizes),
             ("v", v, state, sizes)]
    if bits == 8:
        lists.append(("tops", tops, torch.int32, [-(-k // ADAMW_BLOCK) for k in sizes]))
    if copies is not None:
        lists.append(("copies", copies, torch.bfloat16, sizes))
    for name, tensors, dt, want in lists:
        for i, t in enumerate(tensors):
            if t.dtype != dt or t.numel() != want[i] or t.device != dev:
                raise TypeError(f"{name}[{i}] must be {dt} with {want[i]} elements on {dev}, got "
                                f"{t.dtype}, {t.numel()}, {t.device}")
    if n and not params[0].is_cuda:
        raise TypeError("the library takes device memory: got tensors on " + str(dev))
    at, written = {}, []
    for name, tensors, _, want in lists:
        if not all(t.is_contiguous() for t in tensors):
            raise TypeError(f"{name}: the library takes contiguous tensors")
        at[name] = [t.data_ptr() for t in tensors]
        if name != "grads" and n:
            size = tensors[0].element_size()
            written += [(p, p + k * size, name, i)
                        for i, (p, k) in enumerate(zip(at[name], want)) if k]
    written.sort()
    for x, y in zip(written, written[1:]):
        if y[0] < x[1]:
            raise TypeError(f"{x[2]}[{x[3]}] and {y[2]}[{y[3]}] overlap: one step would write "
                            "them twice")
    ends = [w[1] for w in written]
    for i, p in enumerate(at["grads"]):
        k = bisect.bisect_right(ends, p)
        if sizes[i] and k < len(written) and written[k][0] < p + sizes[i] * grads[i].element_size():
            raise TypeError(f"grads[{i}] overlaps {written[k][2]}[{written[k][3]}], which the step "
                            "writes")
    none = [None] * n
    rows = zip(at["params"], at["grads"], at["m"], at["v"], at.get("tops", none),
               at.get("copies", none), sizes, wd, ls)
    table = (AdamWTensor * max(n, 1))(*[AdamWTensor(*row) for row in rows])
    need = int(LIB.uep_adamw_plan_size(table, n))
    buf = _fresh((max(need, 16),), torch.uint8, dev, stream)
    tiles = ctypes.c_int64(0)
    _check(LIB.uep_adamw_prepare(table, n, pd, gd, bits, _p(buf), buf.numel(),
                                 ctypes.byref(tiles), _s(stream)), "uep_adamw_prepare")
    keep = tuple(tuple(x) for x in (params, grads, m, v, copies or (), tops or ()))
    return AdamWPlan(buf, tiles.value, pd, gd, bits, keep, _s(None).value or 0)


def adamw(plan, step, sched, beta1=0.9, beta2=0.999, eps=1e-8, seed=0, err=None, stream=None):
    """One AdamW step over the plan's tensors, in place.  step: int32 [1] on the device, the
    number of this step (from 1); sched: float32 [2] on the device, the learning rate and a
    factor on every gradient; seed: of the stochastic rounding (8-bit states, bf16 params)."""
    if not isinstance(plan, AdamWPlan):
        raise TypeError("plan must be the AdamWPlan that adamw_prepare returned")
    _buf(step, 1, "step")
    _buf(sched, 2, "sched", torch.float32)
    _buf(err, 1, "err")
    _check(LIB.uep_adamw(_p(plan.buf), plan.n_tiles, plan.param_dtype, plan.grad_dtype,
                         plan.state_bits, _p(step), _p(sched), beta1, beta2, eps,
                         seed & 0xFFFFFFFF, _p(err), _table_stream(plan.buf, plan.home, stream)),
           "uep_adamw")


def adamw_decode(m_codes, v_codes, tops, m=None, v=None, dtype=torch.float32, stream=None):
    """The values of 8-bit AdamW states: m_codes and v_codes uint8 [n] with their `tops` ->
    m, v [n] (float32 or bfloat16, both exact)."""
    n = m_codes.numel()
    _buf(m_codes, n, "m_codes", torch.uint8)
    _buf(v_codes, n, "v_codes", torch.uint8)
    _buf(tops, -(-n // ADAMW_BLOCK), "tops")
    m = _new(m_codes.shape, m_codes, stream, dtype) if m is None else m
    v = _new(m_codes.shape, m_codes, stream, dtype) if v is None else v
    dt = _dtype(m, "m")
    _buf(m, n, "m", m.dtype)
    _buf(v, n, "v", m.dtype)
    _check(LIB.uep_adamw_decode(_p(m_codes), _p(v_codes), _p(tops), n, dt, _p(m), _p(v),
                                _s(stream)), "uep_adamw_decode")
    return m, v


def device_copy(src, dst, stream=None):
    """Plain copy of src into dst (same byte size, both contiguous device tensors)."""
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n or not (src.is_contiguous() and dst.is_contiguous()):
        raise TypeError("device_copy needs two contiguous tensors of the same byte size")
    _check(LIB.uep_device_copy(_p(src), _p(dst), n, _s(stream)), "uep_device_copy")
    return dst


def device_fill(dst, value=0, stream=None):
    """Writes the 32-bit word `value` over the contiguous device tensor dst (a byte size
    that is a multiple of 16)."""
    if not dst.is_contiguous():
        raise TypeError("device_fill needs a contiguous tensor")
    n = dst.numel() * dst.element_size()
    _check(LIB.uep_device_fill(_p(dst), n, value & 0xFFFFFFFF, _s(stream)), "uep_device_fill")
    return dst


def stage_replica_weights(mode, R, E, S, slot_expert, expert_elems, main_w=None, slot_w=None,
                          main_grad=None, slot_grad=None, r_begin=0, r_end=None, stream=None):
    r_end = R if r_end is None else r_end
    n = int(expert_elems)
    _buf(slot_expert, R * S, "slot_expert")
    _buf(main_w, E * n, "main_w", torch.int16)
    _buf(slot_w, R * S * n, "slot_w", torch.int16)
    _buf(main_grad, E * n, "main_grad", torch.float32)
    _buf(slot_grad, R * S * n, "slot_grad", torch.float32)
    _check(LIB.uep_stage_replica_weights(mode, R, E, S, _p(slot_expert), r_begin, r_end,
                                         _p(main_w), _p(slot_w), _p(main_grad), _p(slot_grad),
                                         int(expert_elems), _s(stream)),
           "uep_stage_replica_weights")


def waterfill(counts, topk_ids, batch_size, seed, layer, local_pref_shift=4, shared_rank=None,
              waterline=None, slack=None, rank_load=None, ext_topk=None, want_ext=True,
              stream=None, all_ranks=False):
    _i32(counts, "counts")
    _i32(topk_ids, "topk_ids")
    R, E = counts.shape
    _, T, K = topk_ids.shape
    _buf(batch_size, R, "batch_size")
    shared_rank = _new((R, T), counts, stream) if shared_rank is None \
        else _buf(shared_rank, R * T, "shared_rank")
    waterline = _new((1,), counts, stream) if waterline is None else _buf(waterline, 1, "waterline")
    slack = _new((R,), counts, stream) if slack is None else _buf(slack, R, "slack")
    rank_load = _new((R,), counts, stream) if rank_load is None else _buf(rank_load, R, "rank_load")
    if ext_topk is None and want_ext:
        ext_topk = _new((R, T, K + 1), counts, stream)
    else:
        _buf(ext_topk, R * T * (K + 1), "ext_topk")
    _check(LIB.uep_waterfill(_p(counts), _p(topk_ids), _p(batch_size), R, T, K, E,
                             ctypes.c_uint64(seed & (2 ** 64 - 1)),
                             ctypes.c_uint64(layer & (2 ** 64 - 1)), local_pref_shift,
                             1 if all_ranks else 0, _p(shared_rank), _p(waterline), _p(slack), _p(rank_load),
                             _p(ext_topk), _s(stream)), "uep_waterfill")
    return shared_rank, waterline, slack, rank_load, ext_topk


def lplb_struct_size(R, E, inst_per_rank) -> int:
    return int(LIB.uep_lplb_struct_size(R, E, inst_per_rank))


@dataclasses.dataclass(frozen=True)
class LPStruct:
    """An LP structure from uep_lplb_prepare: the device buffer plus the host's own
    record of its sizes (ranks, experts, instances per rank, instances, replicated
    experts G and their copies n), which the calls below check every caller buffer
    against before a kernel sees it."""

    buf: torch.Tensor
    R: int
    E: int
    inst_per_rank: int
    I: int
    G: int
    n: int
    home: int = 0       # the stream that was current when the buffer was made


def lplb_prepare(inst_expert_host, R, E, inst_per_rank, device, stream=None) -> LPStruct:
    """Offline: build the LP structure from a host instance table into a device buffer."""
    import numpy as np
    ie = np.ascontiguousarray(np.asarray(inst_expert_host, dtype=np.int32))
    if ie.size != R * inst_per_rank:
        raise TypeError(f"inst_expert must have R * inst_per_rank = {R * inst_per_rank} entries")
    n = lplb_struct_size(R, E, inst_per_rank)
    buf = _fresh((max(n, 16),), torch.uint8, device, stream)
    _check(LIB.uep_lplb_prepare(ie.ctypes.data_as(ctypes.c_void_p), R, E, inst_per_rank,
                                _p(buf), buf.numel(), _s(stream)), "uep_lplb_prepare")
    copies = np.bincount(ie[(ie >= 0) & (ie < E)], minlength=E)
    rep = copies >= 2
    return LPStruct(buf, R, E, inst_per_rank, R * inst_per_rank, int(rep.sum()),
                    int(copies[rep].sum()), _s(None).value or 0)


def _lp(lp) -> LPStruct:
    if not isinstance(lp, LPStruct):
        raise TypeError("lp must be the LPStruct that lplb_prepare returned")
    return lp


def lplb(counts, lp, n_copies=None, n_inst=None, iters=30, x=None, m=None, inst_quota=None,
         stats=None, err=None, stream=None):
    """The LP split for one batch.  n_copies and n_inst, when given, must equal the
    structure's own counts; every buffer is checked against the structure."""
    lp = _lp(lp)
    _i32(counts, "counts")
    if tuple(counts.shape) != (lp.R, lp.E):
        raise TypeError(f"counts must be [{lp.R}][{lp.E}] for this LP structure, got "
                        f"{list(counts.shape)}")
    if n_copies is not None and n_copies != lp.n:
        raise TypeError(f"n_copies {n_copies} != the structure's {lp.n} copies")
    if n_inst is not None and n_inst != lp.I:
        raise TypeError(f"n_inst {n_inst} != the structure's {lp.I} instances")
    x = _new((max(lp.n, 1),), counts, stream, torch.float32) if x is None \
        else _buf(x, max(lp.n, 1), "x", torch.float32)
    m = _new((1,), counts, stream, torch.float32) if m is None \
        else _buf(m, 1, "m", torch.float32)
    inst_quota = _new((lp.I,), counts, stream) if inst_quota is None \
        else _buf(inst_quota, lp.I, "inst_quota")
    stats = _new((4,), counts, stream) if stats is None else _buf(stats, 4, "stats")
    _buf(err, 1, "err")
    _check(LIB.uep_lplb(_p(counts), _p(lp.buf), iters, _p(x), _p(m), _p(inst_quota), _p(stats),
                        _p(err), _table_stream(lp.buf, lp.home, stream)), "uep_lplb")
    return x[:lp.n], m, inst_quota, stats


def lplb_plan_workspace_size(R, T, K, E, inst_per_rank) -> int:
    return int(LIB.uep_lplb_plan_workspace_size(R, T, K, E, inst_per_rank))


def lplb_plan(topk_ids, lp, inst_expert, iters=30, r_begin=0, r_end=None, out=None, err=None,
              ws=None, stream=None):
    """uep_lplb_plan: load matrix, LP split and reroute/assignment in one call, with the
    static instance table `inst_expert` [I] the structure was built from.  `out` may hold
    preallocated buffers under the keys below; returns that dict."""
    lp = _lp(lp)
    _i32(topk_ids, "topk_ids")
    R, T, K = topk_ids.shape
    if R != lp.R:
        raise TypeError(f"topk_ids has {R} ranks, the LP structure {lp.R}")
    _buf(inst_expert, lp.I, "inst_expert")
    r_end = R if r_end is None else r_end
    E, I = lp.E, lp.I
    shapes = {"counts": ((R, E), torch.int32), "bucket_pos": ((R, T, K), torch.int32),
              "x": ((max(lp.n, 1),), torch.float32), "m": ((1,), torch.float32),
              "inst_quota": ((I,), torch.int32), "stats": ((4,), torch.int32),
              "xfer": ((R, I), torch.int32), "inst_offset": ((I + 1,), torch.int32),
              "dest_inst": ((R, T, K), torch.int32), "dest_row": ((R, T, K), torch.int32)}
    o = {} if out is None else dict(out)
    for k, (shp, dt) in shapes.items():
        n = 1
        for d in shp:
            n *= d
        o[k] = _new(shp, topk_ids, stream, dt) if o.get(k) is None else _buf(o[k], n, k, dt)
    _buf(err, 1, "err")
    need = lplb_plan_workspace_size(R, T, K, E, lp.inst_per_rank)
    ws = _new((max(need, 4),), topk_ids, stream, torch.uint8) if ws is None else ws
    _check(LIB.uep_lplb_plan(_p(topk_ids), R, T, K, E, _p(lp.buf), lp.inst_per_rank,
                             _p(inst_expert), iters, r_begin, r_end, _p(o["counts"]),
                             _p(o["bucket_pos"]), _p(o["x"]), _p(o["m"]), _p(o["inst_quota"]),
                             _p(o["stats"]), _p(o["xfer"]), _p(o["inst_offset"]),
                             _p(o["dest_inst"]), _p(o["dest_row"]), _p(err), _p(ws),
                             ws.numel() * ws.element_size(),
                             _table_stream(lp.buf, lp.home, stream)), "uep_lplb_plan")
    o["inst_per_rank"] = lp.inst_per_rank
    return o


def lplb_sample(topk_ids, lp, x, seed, layer, dest_inst=None, err=None, stream=None):
    """Per-token copy draw from LPLB's split: dest_inst [R][T][K] int32."""
    lp = _lp(lp)
    _i32(topk_ids, "topk_ids")
    R, T, K = topk_ids.shape
    if R != lp.R:
        raise TypeError(f"topk_ids has {R} ranks, the LP structure {lp.R}")
    _buf(x, lp.n, "x", torch.float32)
    dest_inst = _new((R, T, K), topk_ids, stream) if dest_inst is None \
        else _buf(dest_inst, R * T * K, "dest_inst")
    _buf(err, 1, "err")
    _check(LIB.uep_lplb_sample(_p(topk_ids), R, T, K, _p(lp.buf), _p(x),
                               ctypes.c_uint64(seed & (2 ** 64 - 1)),
                               ctypes.c_uint64(layer & (2 ** 64 - 1)), _p(dest_inst), _p(err),
                               _table_stream(lp.buf, lp.home, stream)), "uep_lplb_sample")
    return dest_inst
