"""Timed cases of the router's balance loss with its gradient, and of the experts' products in
8-bit integers with the rows' way into 8 bits.

Every case runs in two ways on the same inputs: the plain form below (elementary torch
operations, rounded once at the end) and the library's kernels through
``moe_expert_load_amd.uep`` (``own`` true).  ``exact`` states the same operators in 64 bits.
"""

import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


# --------------------------------------------------------------------------- cases
def _balance(op, R, T, E, K, seqs, ragged, score, dtype, add=False):
    """seqs sequences over the R * T tokens, equal or (ragged) with ends anywhere."""
    return {"op": op, "R": R, "T": T, "E": E, "K": K, "seqs": seqs, "ragged": ragged,
            "score": score, "dtype": dtype, "add": add}


def _product(op, rows, experts, n, k, act, skew=0.8):
    """rows over experts (their share falls with rank ** -skew), n outputs of k products."""
    return {"op": op, "rows": rows, "experts": experts, "n": n, "k": k, "act": act, "skew": skew}


def listed():
    return [
        # the small layer of the tests, a sequence per rank
        dict(_balance("balance", 4, 512, 8, 2, 4, False, "softmax", "f32"), name="balance_tiny"),
        # the router of the Qwen3-235B-shaped layer, a loss for each rank's microbatch
        dict(_balance("balance", 32, 8192, 128, 8, 32, False, "softmax", "f32"),
             name="balance_qwen"),
        # DeepSeek-V3-shaped router: sigmoid scores in bf16, packed sequences of any length
        dict(_balance("balance", 64, 4096, 256, 8, 150, True, "sigmoid", "bf16"),
             name="balance_dsv3"),
        # backward of one loss over the Qwen-shaped layer's whole group
        dict(_balance("balance_grad", 32, 8192, 128, 8, 1, False, "softmax", "f32"),
             name="balance_grad_qwen"),
        # backward of the packed sequences, added to the gradient that the gate wrote
        dict(_balance("balance_grad", 64, 4096, 256, 8, 150, True, "sigmoid", "bf16", True),
             name="balance_grad_dsv3"),
        # one decoded token's eight experts of a rank's 32: gate and up products, 7168 wide
        dict(_product("product", 8, 32, 4096, 7168, "swiglu", 0.0), name="product_token"),
        # a decode batch of 128 tokens, skewed: the down products
        dict(_product("product", 1024, 32, 7168, 2048, "plain"), name="product_decode"),
        # odd counts: experts of many, few and no rows, a last step that is not whole
        dict(_product("product", 5003, 13, 1000, 1040, "plain", 1.4), name="product_odd"),
        # prefill on one rank: gate and up products of 4096 tokens' eight experts
        dict(_product("product", 32768, 32, 4096, 7168, "swiglu"), name="product_prefill"),
        # the shared expert on one decoded token, from its bf16 row
        dict(_product("linear", 1, 1, 4096, 7168, "plain"), name="linear_token"),
        # the shared expert on a prefill batch, bf16 rows put into 8 bits first
        dict(_product("linear", 8192, 1, 4096, 4096, "plain"), name="linear_prefill"),
        # 2048 tokens dispatched to eight of 32 experts in 8 bits, gate and up products
        dict(_product("dispatch", 16384, 32, 4096, 4096, "swiglu"), name="dispatch_prefill"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "balance_grad", "product", "product", "linear", "dispatch"])
    if op in ("balance", "balance_grad"):
        E = rng.choice([_log_int(rng, 8, 512), 8 * _log_int(rng, 1, 64)])
        K = min(E, rng.choice([1, 2, 4, 6, 8, 8, 8, 9, 10, 16]))
        R = rng.choice([1, 2, 8, 32])
        T = max(1, _log_int(rng, 1, min(262144, 262144 * 128 // E)) // R)
        ragged = rng.random() < 0.5
        seqs = _log_int(rng, 1, min(200, R * T)) if ragged else rng.choice([1, R])
        return _balance(op, R, T, E, K, seqs, ragged, rng.choice(["softmax", "sigmoid"]),
                        rng.choice(["f32", "bf16"]), op == "balance_grad" and rng.random() < 0.5)
    n, k = 16 * _log_int(rng, 4, 512), 16 * _log_int(rng, 8, 448)
    act = rng.choice(["plain", "swiglu"])
    if op == "linear":
        return _product(op, _log_int(rng, 1, 8192), 1, n, k, act)
    experts = min(_log_int(rng, 1, 64), max(1, (1 << 30) // (n * k)))
    if op == "dispatch":
        return _product(op, min(8, experts) * _log_int(rng, 1, 2048), max(experts, 1), n, k, act,
                        rng.choice([0.0, 0.5, 1.0]))
    return _product(op, _log_int(rng, 1, 32768), experts, n, k, act, rng.choice([0.0, 0.8, 1.4]))


def work(case):
    op = case["op"]
    if op in ("balance", "balance_grad"):
        n = case["R"] * case["T"]
        row = case["E"] * _SIZE[case["dtype"]]
        b = n * (row + 4 * case["K"]) + 8 * case["seqs"] * case["E"]
        if op == "balance_grad":
            b += n * row * (2 if case["add"] else 1)
        return {"bytes": b, "flops": 6 * n * case["E"]}
    rows, n, k = case["rows"], case["n"], case["k"]
    out = n // 2 if case["act"] == "swiglu" else n
    used = sum(c > 0 for c in _counts(case))
    b = used * n * (k + 4) + rows * 2 * out
    if op == "product":
        b += rows * (k + 4)
    else:                                    # a token's bf16 row is read once
        b += rows // min(8, case["experts"]) * 2 * k
    return {"bytes": b, "flops": 2 * rows * n * k}


# --------------------------------------------------------------------------- inputs
def _counts(case):
    """Rows of each expert: they sum to `rows`, the experts' order is the case's own."""
    rows, m = case["rows"], case["experts"]
    if case["op"] == "dispatch":
        return _dispatch(case)[1]
    rng = random.Random(rows * 1_000_003 + m)
    share = [(i + 1.0) ** -case["skew"] for i in range(m)]
    rng.shuffle(share)
    if rows <= m and case["skew"] == 0.0:    # one token's experts: a row for each
        picked = set(rng.sample(range(m), rows))
        return [int(i in picked) for i in range(m)]
    total, ends, s = sum(share), [], 0.0
    for x in share:
        s += x
        ends.append(int(rows * s / total + 0.5))
    ends[-1] = rows
    return [b - a for a, b in zip([0] + ends, ends)]


def _dispatch(case):
    """Experts of every token (distinct, popular ones more often) and the experts' counts."""
    m = case["experts"]
    k = min(8, m)
    tokens = case["rows"] // k
    gen = torch.Generator().manual_seed(case["rows"] * 131 + m)
    lean = -case["skew"] * torch.arange(1, m + 1).log()[torch.randperm(m, generator=gen)]
    u = torch.rand(tokens, m, generator=gen).clamp_(1e-6, 1 - 1e-6)
    ids = torch.topk(lean - torch.log(-torch.log(u)), k, dim=1).indices
    return ids, torch.bincount(ids.reshape(-1), minlength=m).tolist()


def _prepare_balance(case, gen, dev):
    R, T, E, K = case["R"], case["T"], case["E"], case["K"]
    n, G = R * T, case["seqs"]
    lean = 0.8 * torch.randn(E, generator=gen, device=dev)
    logits = (1.3 * torch.randn(n, E, generator=gen, device=dev) + lean).to(_DT[case["dtype"]])
    pull = 0.1 * torch.randn(E, generator=gen, device=dev) if case["score"] == "sigmoid" else 0.0
    ids = torch.topk(torch.sigmoid(logits.float()) + pull, K, dim=-1).indices.to(torch.int32)
    ids[torch.randperm(n, generator=gen, device=dev)[:n // 50]] = -1          # padded tokens
    if case["ragged"]:
        rng = random.Random(n * 31 + G)
        ends = [0] + sorted(rng.randrange(n + 1) for _ in range(G - 1)) + [n - n // 100]
        ends = [min(e, ends[-1]) for e in ends]
    else:
        ends = [n // G * g for g in range(G + 1)]
    s = {"logits": logits.view(R, T, E), "ids": ids.view(R, T, K), "ends": ends, "n_seq": G,
         "offset": torch.tensor(ends, dtype=torch.int32, device=dev) if case["ragged"] else None,
         "score": case["score"], "add": None}
    if case["op"] == "balance":
        s["loss"] = torch.empty(G, device=dev)
        s["counts"] = torch.empty(G, E, dtype=torch.int32, device=dev)
        s["prob"] = torch.empty(G, E, device=dev)
        s["tokens"] = torch.empty(G, dtype=torch.int32, device=dev)
        if own:
            from moe_expert_load_amd import uep as U
            s["ws"] = torch.empty(U.balance_loss_workspace_size(R, T, E, G), dtype=torch.uint8,
                                  device=dev)
        return s
    s["counts"], s["tokens"] = _counted(s, E)
    s["dloss"] = 1e-2 * (0.5 + torch.rand(G, generator=gen, device=dev))
    if case["add"]:
        size = 1e-2 * G / (n * E)            # about that of the loss's own gradient
        s["add"] = (size * torch.randn(n, E, generator=gen, device=dev)).to(_DT[case["dtype"]])
        s["add"] = s["add"].view(R, T, E)
    s["dlogits"] = torch.empty_like(s["logits"])
    return s


def _codes(shape, gen, dev):
    """Integers as rows and weights have them in 8 bits: a bell that the ends cut off."""
    out = torch.empty(shape, dtype=torch.int8, device=dev)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        part = flat[a:a + (1 << 27)]
        part.copy_((36.0 * torch.randn(part.numel(), generator=gen, device=dev)).round_()
                   .clamp_(-127, 127))
    return out


def _prepare_product(case, gen, dev):
    rows, m, n, k = case["rows"], case["experts"], case["n"], case["k"]
    counts = _counts(case)
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    s = {"ends": ends, "act": case["act"], "offset": None,
         "w": _codes((m, n, k), gen, dev),
         "w_scale": 2e-4 * (0.5 + torch.rand(m, n, generator=gen, device=dev))}
    if m > 1:
        s["offset"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    s["out"] = torch.zeros(rows, n // 2 if case["act"] == "swiglu" else n, device=dev,
                           dtype=torch.bfloat16)
    if case["op"] == "product":
        s["q"] = _codes((rows, k), gen, dev)
        s["scale"] = 0.02 * (0.5 + torch.rand(rows, generator=gen, device=dev))
        return s
    s["row"] = None
    tokens = rows
    if case["op"] == "dispatch":
        ids, _ = _dispatch(case)
        tokens = ids.shape[0]
        order = torch.argsort(ids.reshape(-1), stable=True)
        row = torch.empty(rows, dtype=torch.int32)
        row[order] = torch.arange(rows, dtype=torch.int32)
        s["row"] = row.view(1, tokens, -1).to(dev)
    # activations: a few channels are much larger than the others
    loud = 1.0 + 8.0 * (torch.rand(k, generator=gen, device=dev) < 0.01)
    x = torch.randn(tokens, k, generator=gen, device=dev) * loud
    s["x"] = x.to(torch.bfloat16)
    s["q"] = torch.empty(rows, k, dtype=torch.int8, device=dev)
    s["scale"] = torch.empty(rows, device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    make = _prepare_balance if case["op"] in ("balance", "balance_grad") else _prepare_product
    s = make(case, gen, dev)
    s["op"] = case["op"]
    return s


# --------------------------------------------------------------------------- plain forms
def _spans(s):
    return list(zip(s["ends"], s["ends"][1:]))


def _counted(s, E):
    """Ids of every expert and present tokens, for each sequence."""
    K = s["ids"].shape[-1]
    ids = s["ids"].reshape(-1, K)
    counts = [torch.bincount(ids[a:b].reshape(-1).long() + 1, minlength=E + 1)[1:]
              for a, b in _spans(s)]
    tokens = [(ids[a:b] >= 0).any(1).sum() for a, b in _spans(s)]
    return torch.stack(counts).to(torch.int32), torch.stack(tokens).to(torch.int32)


def _shares(s):
    """Scores, and scores that sum to one."""
    x = s["logits"].float()
    x = x.reshape(-1, x.shape[-1])
    if s["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        p = torch.exp(x - x.amax(-1, keepdim=True))
    return x, p / p.sum(-1, keepdim=True)


def _balance_plain(s):
    K = s["ids"].shape[-1]
    _, p = _shares(s)
    E = p.shape[-1]
    counts, tokens = _counted(s, E)
    p = p * (s["ids"].reshape(-1, K) >= 0).any(1, keepdim=True)
    prob = torch.stack([p[a:b].sum(0, dtype=torch.float64) for a, b in _spans(s)])
    n = tokens.double().clamp(min=1).unsqueeze(1)
    prob = prob / n
    loss = (counts * prob).sum(1) * E / (K * n.squeeze(1))
    return [loss.float(), counts, prob.float(), tokens]


def _balance_grad_plain(s):
    K = s["ids"].shape[-1]
    x, p = _shares(s)
    E = p.shape[-1]
    d = torch.zeros_like(p) if s["add"] is None else s["add"].reshape(p.shape).float()
    on = (s["ids"].reshape(-1, K) >= 0).any(1, keepdim=True)
    factor = s["dloss"] * E / (K * s["tokens"].float().clamp(min=1).square())
    for g, (a, b) in enumerate(_spans(s)):
        c = s["counts"][g].float()
        mean = (p[a:b] * c).sum(-1, keepdim=True)
        t = p[a:b] * (c - mean) * factor[g] * on[a:b]
        if s["score"] == "sigmoid":
            t = t / (1.0 + torch.exp(x[a:b]))
        d[a:b] += t
    return d.to(s["logits"].dtype).view_as(s["logits"])


def _rows8_plain(x):
    """Integers and scale of every row; the quotients in 64 bits, where a border's side shows."""
    x = x.float()
    scale = (x.abs().amax(-1) / 127.0).clamp(min=2.0 ** -126)
    return torch.round(x.double() / scale.double().unsqueeze(-1)).to(torch.int8), scale


def _product_plain(s, q, scale):
    out = s["out"]
    for g, (a, b) in enumerate(_spans(s)):
        if a == b:
            continue
        z = q[a:b].float() @ s["w"][g].float().t()
        z = z * s["w_scale"][g] * scale[a:b].unsqueeze(-1)
        if s["act"] == "swiglu":
            gate, up = z.chunk(2, dim=-1)
            z = gate / (1.0 + torch.exp(-gate)) * up
        out[a:b] = z.to(torch.bfloat16)
    return out


def _run_plain(s):
    op = s["op"]
    if op == "balance":
        return _balance_plain(s)
    if op == "balance_grad":
        return _balance_grad_plain(s)
    if op == "product":
        return _product_plain(s, s["q"], s["scale"])
    q, scale = _rows8_plain(s["x"])
    if op == "dispatch":
        k = s["row"].shape[-1]
        token = torch.empty(len(s["scale"]), dtype=torch.int64, device=q.device)
        token[s["row"].reshape(-1).long()] = torch.arange(len(token), device=q.device) // k
        q, scale = q[token], scale[token]
    return _product_plain(s, q, scale)


# --------------------------------------------------------------------------- one pass
def _run_own(s):
    from moe_expert_load_amd import uep as U
    op = s["op"]
    if op in ("balance", "balance_grad"):
        score = U.GATE_SOFTMAX if s["score"] == "softmax" else U.GATE_SIGMOID
        if op == "balance":
            return list(U.balance_loss(s["logits"], s["ids"], n_seq=s["n_seq"],
                                       seq_offset=s["offset"], score=score, loss=s["loss"],
                                       counts=s["counts"], prob=s["prob"], tokens=s["tokens"],
                                       ws=s["ws"]))
        return U.balance_loss_grad(s["dloss"], s["logits"], s["ids"], s["counts"], s["tokens"],
                                   seq_offset=s["offset"], score=score, add=s["add"],
                                   dlogits=s["dlogits"])
    if op == "linear":
        U.quant_rows(s["x"], q=s["q"], scale=s["scale"])
    elif op == "dispatch":
        U.permute_quant(s["x"].unsqueeze(0), s["row"], s["q"], s["scale"])
    act = U.PRODUCT_SWIGLU if s["act"] == "swiglu" else U.PRODUCT_PLAIN
    return U.expert_product(s["q"], s["scale"], s["w"], s["w_scale"], inst_offset=s["offset"],
                            act=act, out=s["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- 64 bits
def _exact_balance(s, op):
    E, K = s["logits"].shape[-1], s["ids"].shape[-1]
    x = s["logits"].double().reshape(-1, E)
    ids = s["ids"].reshape(-1, K).long()
    score = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, -1)
    share = score / score.sum(-1, keepdim=True)
    live = ids.amax(1) >= 0
    picked = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), (ids >= 0).double())
    loss, prob = [], []
    grad = torch.zeros_like(x) if s["add"] is None else s["add"].double().reshape(-1, E)
    for g, (a, b) in enumerate(_spans(s)):
        n = max(1, int(live[a:b].sum()))
        often = picked[a:b].sum(0) * E / (K * n)             # E times the expert's share of ids
        mean = (share[a:b] * live[a:b, None]).sum(0) / n
        loss.append((often * mean).sum())
        prob.append(mean)
        if op == "balance_grad":
            # d loss / d share = often / n, back through the division by the scores' sum, then
            # through the score itself
            up = often.expand(b - a, E) * live[a:b, None] * (float(s["dloss"][g]) / n)
            back = up - (up * share[a:b]).sum(-1, keepdim=True)
            slope = torch.sigmoid(-x[a:b]) if s["score"] == "sigmoid" else 1.0
            grad[a:b] += back * share[a:b] * slope
    if op == "balance_grad":
        return grad.view(s["logits"].shape)
    return [torch.stack(loss), None, torch.stack(prob), None]


def _exact_product(s, op):
    if op == "product":
        q, scale = s["q"].double(), s["scale"].double()
    else:
        x = s["x"].double()
        scale = (x.abs().amax(-1) / 127.0).float().double().clamp(min=2.0 ** -126)
        q = torch.round(x / scale.unsqueeze(-1))
    if op == "dispatch":
        at = s["row"].reshape(-1).long()
        back = torch.empty_like(at)
        back[at] = torch.arange(len(at), device=at.device)
        q = q.repeat_interleave(s["row"].shape[-1], 0)[back]
        scale = scale.repeat_interleave(s["row"].shape[-1])[back]
    parts = []
    for g, (a, b) in enumerate(_spans(s)):
        if b > a:
            z = torch.matmul(q[a:b] * scale[a:b, None],
                             (s["w"][g].double() * s["w_scale"][g].double()[:, None]).t())
            if s["act"] == "swiglu":
                half = z.shape[1] // 2
                z = torch.nn.functional.silu(z[:, :half]) * z[:, half:]
            parts.append(z)
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("balance", "balance_grad"):
        return _exact_balance(s, case["op"])
    return _exact_product(s, case["op"])
