"""Timed cases of the MoE training operators: the router gate and its gradient, the
gradients of dispatch and combine, and the AdamW step.

Every case runs in two ways on the same inputs: the plain form below (elementary torch
operations in 32 bits, rounded once at the end) and the library's kernels through
``moe_expert_load_amd.uep`` (``own`` true).  ``exact`` states the same operators in 64
bits.
"""

import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_BLOCK = 256            # elements that share one window of the 8-bit states
_BETA1, _BETA2, _EPS = 0.9, 0.999, 1e-8


# --------------------------------------------------------------------------- cases
def _gate(op, R, T, E, K, score, renorm, dtype):
    return {"op": op, "R": R, "T": T, "E": E, "K": K, "score": score, "renorm": renorm,
            "dtype": dtype}


def _rows(op, R, T, K, E, H):
    return {"op": op, "R": R, "T": T, "K": K, "E": E, "H": H}


def _adam(tensors, elements, state, param, grad, copy):
    return {"op": "adamw", "tensors": tensors, "elements": elements, "state": state,
            "param": param, "grad": grad, "copy": copy}


def listed():
    return [
        # one decoded token through the router: latency is all that counts
        dict(_gate("gate", 1, 1, 128, 8, "softmax", True, "f32"), name="gate_token"),
        # the router of the Qwen3-235B-shaped layer, the whole group's microbatch
        dict(_gate("gate", 32, 8192, 128, 8, "softmax", True, "f32"), name="gate_qwen"),
        # DeepSeek-V3-shaped router: sigmoid scores, a selection bias, bf16 logits
        dict(_gate("gate", 64, 4096, 256, 8, "sigmoid", True, "bf16"), name="gate_dsv3"),
        # backward of the Qwen-shaped router
        dict(_gate("gate_grad", 32, 8192, 128, 8, "softmax", True, "f32"),
             name="gate_grad_qwen"),
        # an odd expert count with weights that are not renormalised: a dense gradient
        dict(_gate("gate_grad", 3, 4099, 61, 4, "softmax", False, "bf16"),
             name="gate_grad_odd"),
        # the small layer of the tests, backward of the dispatch
        dict(_rows("permute_grad", 4, 512, 2, 8, 256), name="permute_grad_tiny"),
        # 14 KiB rows with the shared-expert column (nine rows a token), ragged tokens
        dict(_rows("permute_grad", 8, 4093, 9, 264, 7168), name="permute_grad_dsv3"),
        # the small layer, backward of the combine
        dict(_rows("combine_grad", 4, 512, 2, 8, 256), name="combine_grad_tiny"),
        # eight ranks of the Qwen-shaped layer: the largest row move of the backward
        dict(_rows("combine_grad", 8, 8192, 8, 128, 4096), name="combine_grad_qwen"),
        # what a layer holds beside its experts: many small and odd tensors
        dict(_adam(96, 1_500_000, 32, "f32", "f32", True), name="adamw_small"),
        # four layers of one rank's experts with fp32 master weights and states
        dict(_adam(16, 16 * 3 * 4096 * 1536, 32, "f32", "f32", True), name="adamw_experts"),
        # the same experts held in bf16 with 8-bit states
        dict(_adam(16, 16 * 3 * 4096 * 1536, 8, "bf16", "bf16", False),
             name="adamw8_experts"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate_grad", "permute_grad", "combine_grad", "adamw", "adamw"])
    if op in ("gate", "gate_grad"):
        E = rng.choice([_log_int(rng, 8, 512), 8 * _log_int(rng, 1, 64)])
        K = min(E, rng.choice([1, 2, 4, 6, 8, 8, 8, 9, 10, 16]))
        R = rng.choice([1, 2, 8, 32])
        most = min(262144, 262144 * 256 // E)
        T = max(1, _log_int(rng, 1, most) // R)
        return _gate(op, R, T, E, K, rng.choice(["softmax", "softmax", "sigmoid"]),
                     rng.random() < 0.6, rng.choice(["f32", "bf16"]))
    if op in ("permute_grad", "combine_grad"):
        R, K = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8, 8, 9])
        E = R * rng.choice([3, 16, 32])
        H = 8 * _log_int(rng, 16, 1024)
        T = max(1, _log_int(rng, 1, max(2, min(65536, (1 << 31) // (K * H)))) // R)
        return _rows(op, R, T, min(K, E), E, H)
    state = rng.choice([8, 32])
    param = rng.choice(["f32", "bf16"])
    return _adam(_log_int(rng, 1, 200), _log_int(rng, 20_000, 250_000_000), state, param,
                 rng.choice(["f32", "bf16"]), param == "f32" and rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "adamw":
        n, p, g = sum(_sizes(case)), _SIZE[case["param"]], _SIZE[case["grad"]]
        b = n * (2 * p + g + (2 if case["copy"] else 0))
        # 8-bit states are read back as bf16 values too (two codes read, two values written)
        b += n * (2 * 8 if case["state"] == 32 else 2 * 2 + 2 + 2 * 2)
        return {"bytes": b, "flops": 16 * n}
    n = case["R"] * case["T"]
    if op in ("gate", "gate_grad"):
        row = case["E"] * _SIZE[case["dtype"]]
        b = n * (row + 8 * case["K"])
        if op == "gate_grad":
            dense = case["score"] == "softmax" and not case["renorm"]
            picked = case["score"] == "sigmoid" and case["renorm"]
            b += n * (4 * case["K"] + (row if dense else 0)
                      + (case["K"] * _SIZE[case["dtype"]] if picked else 0))
        return {"bytes": b, "flops": 4 * n * case["E"]}
    rows, H = n * case["K"], case["H"]
    if op == "permute_grad":
        return {"bytes": (rows + n) * H * 2 + rows * 4, "flops": rows * H}
    return {"bytes": (2 * rows + n) * H * 2 + rows * 12, "flops": 3 * rows * H}


# --------------------------------------------------------------------------- inputs
def _sizes(case):
    """Element counts of the case's tensors: equal blocks where they divide evenly, else a
    spread over two orders of magnitude with odd lengths."""
    c, n = case["tensors"], case["elements"]
    if n % (c * 4096) == 0:
        return [n // c] * c
    rng = random.Random(c * 1_000_003 + n)
    w = [math.exp(rng.uniform(0.0, 4.6)) for _ in range(c)]
    s = sum(w)
    return [max(1, int(n * x / s)) for x in w]


def _routing(gen, n, K, E, dev):
    """Distinct expert ids per token, Zipf popularity, 2 % of the tokens absent (-1)."""
    pop = torch.arange(1, E + 1, device=dev, dtype=torch.float32).pow(-0.8).log()
    pop = pop[torch.randperm(E, generator=gen, device=dev)]
    u = torch.rand(n, E, generator=gen, device=dev).clamp_(1e-7, 1 - 1e-7)
    ids = torch.topk(pop - torch.log(-torch.log(u)), K, dim=1).indices
    ids[torch.randperm(n, generator=gen, device=dev)[:n // 50]] = -1
    return ids


def _far_apart(logits, bias, K):
    """Rows in which two of the best K + 1 selection scores are closer than fp32 can tell
    apart get the logits of a row in which they are not."""
    key = torch.sigmoid(logits.double()) + bias.double()
    top = torch.topk(key, min(K + 1, key.shape[-1]), dim=-1).values
    if top.shape[-1] > 1:
        bad = (top[:, :-1] - top[:, 1:]).amin(-1) < 2e-6
        good = torch.nonzero(~bad)
        if len(good):
            logits[bad] = logits[good[0, 0]].clone()
    return logits


def _prepare_gate(case, gen, dev):
    R, T, E, K = case["R"], case["T"], case["E"], case["K"]
    n = R * T
    lean = 0.8 * torch.randn(E, generator=gen, device=dev)
    logits = (1.3 * torch.randn(n, E, generator=gen, device=dev) + lean).to(_DT[case["dtype"]])
    s = {"K": K, "bias": None, "score": case["score"], "renorm": case["renorm"],
         "scale": 2.5 if case["score"] == "sigmoid" else 1.0}
    if case["score"] == "sigmoid":
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device=dev)
        logits = _far_apart(logits, s["bias"], K)
    s["logits"] = logits.view(R, T, E)
    s["ids"] = torch.empty(R, T, K, dtype=torch.int32, device=dev)
    s["w"] = torch.empty(R, T, K, dtype=torch.float32, device=dev)
    if case["op"] == "gate_grad":
        s["ids"], s["w"] = _gate_plain(s)
        s["dw"] = torch.randn(R, T, K, generator=gen, device=dev)
        s["dlogits"] = torch.empty_like(s["logits"])
    return s


def _prepare_rows(case, gen, dev):
    R, T, K, E, H = (case[k] for k in ("R", "T", "K", "E", "H"))
    n = R * T
    flat = _routing(gen, n, K, E, dev).reshape(-1)
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    row = torch.empty(n * K, dtype=torch.int64, device=dev)
    row[order] = torch.arange(n * K, device=dev)
    row[flat < 0] = -1
    P = int((flat >= 0).sum())
    bf = torch.bfloat16
    s = {"row": row.to(torch.int32).view(R, T, K), "P": P}
    if case["op"] == "permute_grad":
        s["dout"] = torch.randn(P, H, generator=gen, device=dev, dtype=bf)
        s["dx"] = torch.empty(R, T, H, device=dev, dtype=bf)
        return s
    s["dy"] = torch.randn(R, T, H, generator=gen, device=dev, dtype=bf)
    s["out"] = torch.randn(P, H, generator=gen, device=dev, dtype=bf)
    s["w"] = torch.softmax(torch.randn(R, T, K, generator=gen, device=dev), -1)
    s["dout"] = torch.empty(P, H, device=dev, dtype=bf)
    s["dw"] = torch.empty(R, T, K, device=dev)
    return s


def _prepare_adamw(case, gen, dev):
    sizes = _sizes(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // _BLOCK) * _BLOCK
    live = torch.zeros(at, dtype=torch.bool, device=dev)
    for a, n in zip(starts, sizes):
        live[a:a + n] = True
    spread = torch.exp(1.5 * torch.randn(at, generator=gen, device=dev))
    g = torch.randn(at, generator=gen, device=dev) * spread * 1e-3 * live
    m = (0.3 * torch.randn(at, generator=gen, device=dev) * spread * 1e-3) * live
    v = (spread * 1e-3).square() * (0.5 + torch.rand(at, generator=gen, device=dev)) * live
    del spread
    p = (0.02 * torch.randn(at, generator=gen, device=dev) * live).to(_DT[case["param"]])
    s = {"starts": starts, "sizes": sizes, "p": p, "g": g.to(_DT[case["grad"]]),
         "copy": p.to(torch.bfloat16) if case["copy"] else None, "state": case["state"],
         "decay": [0.1 if i % 3 else 0.0 for i in range(len(sizes))],
         "step": torch.full((1,), 137, dtype=torch.int32, device=dev),
         "sched": torch.tensor([3e-4, 0.7], device=dev), "seed": int(case["elements"]) & 0xFFFF}
    if case["state"] == 32:
        s["m"], s["v"], s["tops"] = m, v, None
    else:
        half = torch.full((1,), 1 << 15, dtype=torch.int64, device=dev)
        s["m"], mt = _encode(m, half, 127)
        s["v"], vt = _encode(v, half, 255)
        s["tops"] = (mt | (vt << 16)).to(torch.int32)
        s["m_value"] = torch.empty(at, dtype=torch.bfloat16, device=dev)
        s["v_value"] = torch.empty(at, dtype=torch.bfloat16, device=dev)
    return s


def _parts(s, key):
    return [s[key][a:a + n] for a, n in zip(s["starts"], s["sizes"])]


def _tops(s):
    return [s["tops"][a // _BLOCK:(a + n + _BLOCK - 1) // _BLOCK]
            for a, n in zip(s["starts"], s["sizes"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if case["op"] in ("gate", "gate_grad"):
        s = _prepare_gate(case, gen, dev)
    elif case["op"] in ("permute_grad", "combine_grad"):
        s = _prepare_rows(case, gen, dev)
    else:
        s = _prepare_adamw(case, gen, dev)
        if own:               # the table of tensors a training program makes once
            from moe_expert_load_amd import uep as U
            s["plan"] = U.adamw_prepare(
                _parts(s, "p"), _parts(s, "g"), _parts(s, "m"), _parts(s, "v"),
                copies=_parts(s, "copy") if case["copy"] else None,
                tops=_tops(s) if case["state"] == 8 else None, weight_decay=s["decay"])
    s["op"] = case["op"]
    return s


# --------------------------------------------------------------------------- plain forms
def _gate_plain(s):
    x = s["logits"].float()
    able = torch.isfinite(x)
    score = torch.exp(x - x.amax(-1, keepdim=True)) if s["score"] == "softmax" else \
        1.0 / (1.0 + torch.exp(-x))
    key = x if s["score"] == "softmax" else score + s["bias"]
    key, order = torch.sort(key.masked_fill(~able, -math.inf), dim=-1, descending=True,
                            stable=True)
    ids, none = order[..., :s["K"]], key[..., :s["K"]] == -math.inf
    w = score.masked_fill(~able, 0.0)
    total = w.sum(-1, keepdim=True)
    w = w.gather(-1, ids).masked_fill(none, 0.0)
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
    if s["renorm"] or s["score"] == "softmax":
        w = w / total
    return ids.masked_fill(none, -1).to(torch.int32), w * s["scale"]


def _gate_grad_plain(s):
    x, scale = s["logits"].float(), s["scale"]
    at, on = s["ids"].clamp(min=0).long(), s["ids"] >= 0
    g, u = s["dw"] * scale * on, s["w"] / scale
    if s["renorm"]:
        d = u * (g - (u * g).sum(-1, keepdim=True))
        if s["score"] == "sigmoid":
            d = d * (1.0 - 1.0 / (1.0 + torch.exp(-x.gather(-1, at))))
        d = torch.zeros_like(x).scatter_add_(-1, at, d * on)
    elif s["score"] == "sigmoid":
        d = torch.zeros_like(x).scatter_add_(-1, at, u * (1.0 - u) * g)
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        e = e / e.sum(-1, keepdim=True)
        pick = torch.zeros_like(x).scatter_add_(-1, at, g)
        d = e * (pick - (u * g).sum(-1, keepdim=True))
    return d.to(s["logits"].dtype)


def _permute_grad_plain(s):
    R, T, K = s["row"].shape
    row = s["row"].reshape(R * T, K)
    d = s["dout"].float()[row.clamp(min=0)] * (row >= 0).unsqueeze(-1)
    return d.sum(1).to(torch.bfloat16).view(R, T, -1)


def _combine_grad_plain(s):
    R, T, K = s["row"].shape
    row = s["row"].reshape(-1)
    on = torch.nonzero(row >= 0).squeeze(-1)
    rows = row[on].long()
    dy = s["dy"].view(R * T, -1).float()[on // K]
    dw = torch.zeros(R * T * K, device=row.device)
    dw[on] = (dy * s["out"].float()[rows]).sum(-1)
    s["dout"][rows] = (dy * s["w"].reshape(-1)[on].unsqueeze(-1)).to(torch.bfloat16)
    return [s["dout"], dw.view(R, T, K)]


def _words(seed, step, tensor, n, dev):
    """Random bits of one tensor's elements: six 32-bit words for each group of four."""
    def mix(x):
        x = x ^ (x >> 16)
        x = (x * 0x9E3779B9) & 0xFFFFFFFF
        x = x ^ (x >> 15)
        x = (x * 0xBB67AE85) & 0xFFFFFFFF
        return x ^ (x >> 16)

    def shift(x):
        x = x ^ ((x << 13) & 0xFFFFFFFF)
        x = x ^ (x >> 17)
        return x ^ ((x << 5) & 0xFFFFFFFF)

    key = mix(mix((step.long() * 0x9E3779B9 + seed) & 0xFFFFFFFF) ^ (tensor + 1))
    w0 = mix(((torch.arange(-(-n // 4), device=dev) * 0x9E3779B9) & 0xFFFFFFFF) ^ key)
    w1 = shift(w0)
    w2 = shift(w1)
    w3 = shift(w2)
    w4 = shift(w3)
    param = torch.stack([w0 & 0xFFFF, w0 >> 16, w1 & 0xFFFF, w1 >> 16], 1).reshape(-1)[:n]
    state = torch.stack([w2, w3, w4, shift(w4)], 1).reshape(-1)[:n]
    return param, state


def _encode(x, dither, span):
    """Codes and top level of every block of 256: the float's upper bits (8 of exponent, 3 of
    mantissa), rounded by `dither` / 2**16, counted down from the block's largest."""
    n = x.numel()
    bits = x.abs().view(torch.int32).long()
    level = ((bits + (dither << 4)) >> 20).clamp(max=0x7F7)
    level = torch.where(bits > 0, level, 0)
    padded = torch.nn.functional.pad(level, (0, -n % _BLOCK)).view(-1, _BLOCK)
    top = padded.amax(1)
    code = (padded - top.unsqueeze(1) + span).view(-1)[:n]
    if span == 255:           # a second moment above zero never becomes zero
        code = torch.where(bits > 0, code.clamp(min=1), 0)
    else:
        code = torch.where(bits > 0, code.clamp(min=0), 0)
        code = torch.where(code > 0, code | ((x < 0).long() << 7), 0)
    return code.to(torch.uint8), top


def _decode(code, tops, span):
    n = code.numel()
    c = code.long()
    top = tops.long() & 0xFFFF if span == 127 else tops.long() >> 16
    size = c & span
    level = (size - span + top.repeat_interleave(_BLOCK)[:n]).clamp(min=0)
    x = (torch.where(size > 0, level, 0) << 20).to(torch.int32).view(torch.float32)
    return torch.where(c > 127, -x, x) if span == 127 else x


def _adamw_tensor(s, i, p, g, m, v, tops, copy):
    n, eight = p.numel(), s["state"] == 8
    step, (lr, scale) = s["step"].double(), s["sched"]
    c1, c2 = (1.0 - _BETA1 ** step).float(), (1.0 - _BETA2 ** step).float()
    grad = g.float() * scale
    m1 = (_decode(m, tops, 127) if eight else m) * _BETA1 + grad * (1.0 - _BETA1)
    v1 = (_decode(v, tops, 255) if eight else v) * _BETA2 + grad * grad * (1.0 - _BETA2)
    w = p.float() * (1.0 - lr * s["decay"][i]) \
        - (lr / c1) * (m1 / (torch.sqrt(v1) / torch.sqrt(c2) + _EPS))
    if eight or p.dtype == torch.bfloat16:
        for_p, for_s = _words(s["seed"], s["step"], i, n, p.device)
    if eight:
        code, mt = _encode(m1, for_s & 0xFFFF, 127)
        m.copy_(code)
        code, vt = _encode(v1, for_s >> 16, 255)
        v.copy_(code)
        tops.copy_(mt | (vt << 16))
    else:
        m.copy_(m1)
        v.copy_(v1)
    if p.dtype == torch.bfloat16:
        w = ((w.view(torch.int32) + for_p.to(torch.int32)) & -65536).view(torch.float32)
    p.copy_(w)
    if copy is not None:
        copy.copy_(w)


def _adamw_plain(s):
    eight = s["state"] == 8
    parts = [_parts(s, k) for k in ("p", "g", "m", "v")]
    none = [None] * len(s["sizes"])
    tops = _tops(s) if eight else none
    copies = _parts(s, "copy") if s["copy"] is not None else none
    list(map(lambda i: _adamw_tensor(s, i, *(x[i] for x in parts), tops[i], copies[i]),
             range(len(s["sizes"]))))
    if eight:
        s["m_value"].copy_(_decode(s["m"], s["tops"], 127))
        s["v_value"].copy_(_decode(s["v"], s["tops"], 255))


# --------------------------------------------------------------------------- one pass
def _run_own(s):
    from moe_expert_load_amd import uep as U
    op = s["op"]
    if op in ("gate", "gate_grad"):
        score = U.GATE_SOFTMAX if s["score"] == "softmax" else U.GATE_SIGMOID
        if op == "gate":
            return list(U.gate(s["logits"], s["K"], bias=s["bias"], score=score,
                               renorm=s["renorm"], scale=s["scale"], topk_ids=s["ids"],
                               gate_w=s["w"]))
        return U.gate_grad(s["dw"], s["logits"], s["ids"], s["w"], score=score,
                           renorm=s["renorm"], scale=s["scale"], dlogits=s["dlogits"])
    if op == "permute_grad":
        return U.permute_grad(s["dout"], s["row"], s["dx"])
    if op == "combine_grad":
        return list(U.combine_grad(s["dy"], s["out"], s["row"], s["w"], s["dout"], s["dw"]))
    U.adamw(s["plan"], s["step"], s["sched"], beta1=_BETA1, beta2=_BETA2, eps=_EPS,
            seed=s["seed"])
    if s["state"] == 8:
        U.adamw_decode(s["m"], s["v"], s["tops"], s["m_value"], s["v_value"])
    return None


def run(state):
    op = state["op"]
    if own:
        got = _run_own(state)
    elif op == "gate":
        got = list(_gate_plain(state))
    elif op == "gate_grad":
        got = _gate_grad_plain(state)
    elif op == "permute_grad":
        got = _permute_grad_plain(state)
    elif op == "combine_grad":
        got = _combine_grad_plain(state)
    else:
        got = _adamw_plain(state)
    if op != "adamw":
        return got
    held = ("m", "v") if state["state"] == 32 else ("m_value", "v_value")
    return [state["p"], state[held[0]], state[held[1]]] + \
        ([state["copy"]] if state["copy"] is not None else [])


# --------------------------------------------------------------------------- 64 bits
def _exact_gate(s, op):
    x = s["logits"].double()
    soft = s["score"] == "softmax"
    p = torch.softmax(x, -1) if soft else torch.sigmoid(x)
    key = x if soft else p + s["bias"].double()
    ids = s["ids"].long() if op == "gate_grad" else \
        torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :s["K"]]
    w = p.gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    if op == "gate":
        return [None, w * s["scale"]]
    # chain rule through the weights, one Jacobian-vector product at a time
    dw = s["dw"].double() * s["scale"]
    if s["renorm"]:
        total = p.gather(-1, ids).sum(-1, keepdim=True)
        dsel = (dw - (dw * w).sum(-1, keepdim=True)) / total
    else:
        dsel = dw
    dp = torch.zeros_like(p).scatter_(-1, ids, dsel)
    if soft:
        return p * (dp - (dp * p).sum(-1, keepdim=True))
    return p * (1.0 - p) * dp


def _exact_rows(s, op):
    R, T, K = s["row"].shape
    n = R * T
    row = s["row"].reshape(n, K).long()
    H = (s["dout"] if op == "permute_grad" else s["dy"]).shape[-1]
    if op == "permute_grad":
        dx = torch.zeros(n, H, dtype=torch.float64, device=row.device)
        for k in range(K):
            on = row[:, k] >= 0
            dx[on] += s["dout"][row[on, k]].double()
        return dx.view(R, T, H)
    dout = torch.zeros(s["P"], H, dtype=torch.float64, device=row.device)
    dw = torch.zeros(n, K, dtype=torch.float64, device=row.device)
    dy = s["dy"].view(n, H)
    for k in range(K):
        on = torch.nonzero(row[:, k] >= 0).squeeze(-1)
        d = dy[on].double()
        dw[on, k] = (d * s["out"][row[on, k]].double()).sum(-1)
        dout[row[on, k]] = d * s["w"].view(n, K)[on, k].double().unsqueeze(-1)
    return [dout, dw.view(R, T, K)]


def _level64(x, dither):
    """Where x lies on the ladder of floats with three bits of mantissa, rounded down after
    `dither` / 2**16 of a step was added."""
    mant, ex = torch.frexp(x)
    at = (ex.double() + 126.0) * 8.0 + (2.0 * mant - 1.0) * 8.0
    return torch.where(x > 0, torch.floor(at + dither.double() / 65536.0), 0.0)


def _exact_state(x, dither, span):
    n = x.numel()
    level = _level64(x.abs(), dither)
    padded = torch.nn.functional.pad(level, (0, -n % _BLOCK)).view(-1, _BLOCK)
    low = (padded.amax(1, keepdim=True) - span).expand(-1, _BLOCK).reshape(-1)[:n]
    floor = torch.maximum(level, low + 1) if span == 255 else level
    return torch.where((x != 0) & (floor > low), _value64(floor), 0.0) * torch.sign(x)


def _value64(level):
    y = torch.exp2(torch.floor(level / 8.0) - 127.0) * (1.0 + torch.remainder(level, 8.0) / 8.0)
    return torch.where(level > 0, y, 0.0)


def _held64(s, key):
    """What the 8-bit states stand for, from the codes' definition."""
    span, code = (127, s[key] & 127) if key == "m" else (255, s[key])
    top = s["tops"] % 65536 if key == "m" else s["tops"] // 65536
    level = code.double() + top.double().repeat_interleave(_BLOCK)[:code.numel()] - span
    y = torch.where(code > 0, _value64(level), 0.0)
    return torch.where(s[key] >= 128, -y, y) if key == "m" else y


def _exact_adamw(s):
    eight = s["state"] == 8
    lr, scale = (float(x) for x in s["sched"].tolist())
    t = int(s["step"].item())
    got = [torch.zeros(s["p"].numel(), dtype=torch.float64, device=s["p"].device)
           for _ in range(3)]
    mv = [_held64(s, "m"), _held64(s, "v")] if eight else [s["m"], s["v"]]
    for i, (a, n) in enumerate(zip(s["starts"], s["sizes"])):
        at = slice(a, a + n)
        g = s["g"][at].double() * scale
        m = _BETA1 * mv[0][at].double() + (1 - _BETA1) * g
        v = _BETA2 * mv[1][at].double() + (1 - _BETA2) * g * g
        hat = (m / (1 - _BETA1 ** t)) / (torch.sqrt(v / (1 - _BETA2 ** t)) + _EPS)
        p = s["p"][at].double()
        got[0][at] = p - lr * s["decay"][i] * p - lr * hat
        if eight:
            _, r = _words(s["seed"], s["step"], i, n, p.device)
            m, v = _exact_state(m, r & 0xFFFF, 127), _exact_state(v, r >> 16, 255)
        got[1][at], got[2][at] = m, v
    return got + ([got[0]] if s["copy"] is not None else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gate", "gate_grad"):
        return _exact_gate(s, case["op"])
    if case["op"] in ("permute_grad", "combine_grad"):
        return _exact_rows(s, case["op"])
    return _exact_adamw(s)
