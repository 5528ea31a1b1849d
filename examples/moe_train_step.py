"""One MoE layer trained through the library: every step of the layer that is not a plain
matrix product runs in its kernels.  Once trained it also answers in 8 bits, products and all.

    router logits -> gate -> plan (replicas, quotas, rows) -> replica weights staged ->
    permute -> experts -> combine -> loss (and the router's balance loss, a sequence per rank)
    loss -> combine gradient -> experts' backward -> replica gradients reduced ->
    permute gradient, gate gradient, balance gradient -> AdamW over the experts and the router
    8 bits: ... plan -> replica weights staged -> dispatch in 8 bits -> gate and up products ->
    rows to 8 bits -> down products -> combine

The layer's ranks are virtual, as everywhere in this library; an instance of an expert (its
main, or a replica in a redundant slot) computes on the rows that the plan gave it.  The
experts are SwiGLU blocks (gate, up and down matrices) held in bf16 beside fp32 master
weights; in training their matrix products are torch's, in fp32.

    python examples/moe_train_step.py --steps 30 --state-bits 8 --balance 0.01
"""

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_expert_load_amd import uep as U    # noqa: E402


@dataclasses.dataclass
class Geometry:
    R: int = 4          # ranks
    T: int = 256        # tokens per rank
    K: int = 2          # experts per token
    E: int = 8          # experts
    S: int = 1          # redundant slots per rank
    H: int = 128        # hidden size
    F: int = 64         # an expert's inner size
    q_min: int = 16     # smallest quota of a replica
    balance: float = 0.0    # weight of the balance loss


class Layer:
    """Weights, gradients, optimizer state and buffers of the layer."""

    def __init__(self, geo, seed=0, state_bits=32, lr=2e-3, device="cuda"):
        self.geo = g = geo
        gen = torch.Generator(device=device).manual_seed(seed)
        self.n = 3 * g.H * g.F                                   # elements of an expert
        self.master = 0.1 * torch.randn(g.E, self.n, generator=gen, device=device)
        self.main_w = self.master.to(torch.bfloat16)
        self.main_grad = torch.zeros_like(self.master)
        self.slot_w = torch.zeros(g.R, g.S, self.n, device=device, dtype=torch.bfloat16)
        self.slot_grad = torch.zeros(g.R, g.S, self.n, device=device)
        # skewed on purpose: the first experts are the popular ones
        self.router = 0.3 * torch.randn(g.H, g.E, generator=gen, device=device)
        self.router_grad = torch.zeros_like(self.router)
        self.lean = torch.linspace(1.5, -1.5, g.E, device=device)
        params = [self.master, self.router]
        kind = torch.float32 if state_bits == 32 else torch.uint8
        m, v = ([torch.zeros(p.shape, dtype=kind, device=device) for p in params]
                for _ in range(2))
        tops = None if state_bits == 32 else [
            torch.zeros(-(-p.numel() // U.ADAMW_BLOCK), dtype=torch.int32, device=device)
            for p in params]
        self.router_copy = self.router.to(torch.bfloat16)
        self.adam = U.adamw_prepare(params, [self.main_grad, self.router_grad], m, v,
                                    copies=[self.main_w, self.router_copy], tops=tops,
                                    weight_decay=[0.01, 0.0])
        self.step = torch.zeros(1, dtype=torch.int32, device=device)
        self.sched = torch.tensor([lr, 1.0], device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def _matrices(self, flat):
        g = self.geo
        gate, up, down = flat.float().view(3, g.H * g.F)
        return gate.view(g.H, g.F), up.view(g.H, g.F), down.view(g.F, g.H)

    def _instances(self, plan):
        """(first row, last row, weights, gradients) of every instance with rows."""
        g, ipr = self.geo, plan["inst_per_rank"]
        first = plan["inst_offset"].tolist()
        expert = plan["inst_expert"].tolist()
        for i, e in enumerate(expert):
            if e < 0 or first[i] == first[i + 1]:
                continue
            r, j = divmod(i, ipr)
            slot = j - g.E // g.R
            w, dw = (self.main_w[e], self.main_grad[e]) if slot < 0 else \
                (self.slot_w[r, slot], self.slot_grad[r, slot])
            yield first[i], first[i + 1], w, dw

    def forward(self, x):
        """y [R][T][H] bf16 for x [R][T][H] bf16, and what backward needs."""
        g = self.geo
        logits = x.float() @ self.router + self.lean
        ids, w = U.gate(logits, g.K, err=self.err)
        plan = U.plan(ids, g.E, g.S, g.q_min, err=self.err)
        slots = plan["slot_expert"]
        U.stage_replica_weights(U.STAGE_WEIGHTS, g.R, g.E, g.S, slots, self.n,
                                main_w=self.main_w, slot_w=self.slot_w)
        rows = torch.zeros(g.R * g.T * g.K, g.H, dtype=torch.bfloat16, device=x.device)
        U.permute(x, plan["dest_row"], rows, err=self.err)
        out = torch.zeros_like(rows)
        for a, b, weights, _ in self._instances(plan):
            gate, up, down = self._matrices(weights)
            h = rows[a:b].float()
            out[a:b] = ((torch.nn.functional.silu(h @ gate) * (h @ up)) @ down).to(out.dtype)
        y = torch.empty_like(x)
        U.combine(out, plan["dest_row"], w, y, err=self.err)
        return y, (x, logits, ids, w, plan, rows, out)

    def backward(self, dy, saved):
        """Gradients of the experts and the router for dy [R][T][H] bf16; returns dx in fp32."""
        g = self.geo
        x, logits, ids, w, plan, rows, out = saved
        drow = plan["dest_row"]
        self.main_grad.zero_()
        dout, dgate_w = U.combine_grad(dy, out, drow, w, out, err=self.err)   # in place
        drows = torch.zeros_like(rows)
        for a, b, weights, grad in self._instances(plan):
            gate, up, down = self._matrices(weights)
            h, d = rows[a:b].float(), dout[a:b].float()
            p, q = h @ gate, h @ up
            s = torch.sigmoid(p)
            dz = d @ down.t()
            dp, dq = dz * q * s * (1 + p * (1 - s)), dz * p * s
            grad += torch.cat([(h.t() @ dp).view(-1), (h.t() @ dq).view(-1),
                               ((p * s * q).t() @ d).view(-1)])
            drows[a:b] = (dp @ gate.t() + dq @ up.t()).to(drows.dtype)
        U.stage_replica_weights(U.STAGE_GRAD_REDUCE, g.R, g.E, g.S, plan["slot_expert"], self.n,
                                main_grad=self.main_grad, slot_grad=self.slot_grad)
        dx = torch.empty_like(x)
        U.permute_grad(drows, drow, dx, err=self.err)
        dlogits = U.gate_grad(dgate_w, logits, ids, w, err=self.err)
        if g.balance:
            _, counts, _, tokens = self.balance_loss(logits, ids)
            each = torch.full((g.R,), g.balance / g.R, device=x.device)
            U.balance_loss_grad(each, logits, ids, counts, tokens, add=dlogits, dlogits=dlogits,
                                err=self.err)
        flat = dlogits.view(-1, g.E)
        torch.matmul(x.view(-1, g.H).float().t(), flat, out=self.router_grad)
        return dx.float() + (flat @ self.router.t()).view_as(x)

    def balance_loss(self, logits, ids):
        """(loss, counts, mean scores, tokens) of every rank's tokens as a sequence."""
        return U.balance_loss(logits, ids, n_seq=self.geo.R, err=self.err)

    def quantise(self):
        """The experts in 8 bits, a scale for each output channel: gates and ups [E][2F][H], downs
        [E][H][F]."""
        g = self.geo
        gate, up, down = zip(*(self._matrices(w) for w in self.main_w))
        pairs = ([torch.cat([a.t(), b.t()]) for a, b in zip(gate, up)], [d.t() for d in down])
        self.int8 = []
        for mats in pairs:
            m = torch.stack(mats).to(torch.bfloat16).contiguous()
            q, scale = U.quant_rows(m.view(-1, m.shape[-1]), err=self.err)
            self.int8.append((q.view(m.shape), scale.view(m.shape[:2]),
                              q.new_zeros(g.R, g.S, *m.shape[1:]),
                              scale.new_zeros(g.R, g.S, m.shape[1])))

    def forward_int8(self, x):
        """y [R][T][H] bf16 for x [R][T][H] bf16 with the experts of the last quantise()."""
        g = self.geo
        logits = x.float() @ self.router + self.lean
        ids, w = U.gate(logits, g.K, err=self.err)
        plan = U.plan(ids, g.E, g.S, g.q_min, err=self.err)
        drow, off = plan["dest_row"], plan["inst_offset"]
        for main, scale, slot, slot_scale in self.int8:
            for a, b in ((main, slot), (scale, slot_scale)):
                a, b = a.view(torch.int16), b.view(torch.int16)
                U.stage_replica_weights(U.STAGE_WEIGHTS, g.R, g.E, g.S, plan["slot_expert"],
                                        a.numel() // g.E, main_w=a, slot_w=b)
        P = g.R * g.T * g.K
        q = torch.zeros(P, g.H, dtype=torch.int8, device=x.device)
        scale = torch.zeros(P, device=x.device)
        U.permute_quant(x, drow, q, scale, err=self.err)
        for (main, main_scale, slot, slot_scale), act in zip(
                self.int8, (U.PRODUCT_SWIGLU, U.PRODUCT_PLAIN)):
            if act == U.PRODUCT_PLAIN:
                q, scale = U.quant_rows(out, live_rows=off[-1:], err=self.err)
            out = U.expert_product(q, scale, main, main_scale, off, g.R, g.S, slot, slot_scale,
                                   act=act, err=self.err)
        y = torch.empty_like(x)
        U.combine(out, drow, w, y, err=self.err)
        return y

    def update(self):
        self.step += 1
        U.adamw(self.adam, self.step, self.sched, seed=1, err=self.err)

    def train_step(self, x, target):
        """One step on the mean squared error; returns the loss (a device scalar)."""
        y, saved = self.forward(x)
        diff = y.float() - target
        dy = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        self.backward(dy, saved)
        self.update()
        return diff.square().mean()


def train(steps=30, seed=0, state_bits=32, geo=None):
    """Losses of `steps` steps on fixed random data."""
    return fit(Layer(geo or Geometry(), seed, state_bits), steps, seed)[0]


def fit(layer, steps, seed):
    """Losses of `steps` steps of a layer on fixed random data, and the data."""
    g = layer.geo
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(g.R, g.T, g.H, generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.tanh(x.float() @ (0.2 * torch.randn(g.H, g.H, generator=gen, device="cuda")))
    losses = [layer.train_step(x, target) for _ in range(steps)]
    losses = [float(v) for v in losses]
    if int(layer.err.item()):
        raise RuntimeError(f"the library reported error bits {int(layer.err.item())}")
    return losses, x


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--balance", type=float, default=0.0, help="weight of the balance loss")
    a = ap.parse_args()
    layer = Layer(Geometry(balance=a.balance), a.seed, a.state_bits)
    losses, x = fit(layer, a.steps, a.seed)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i + 1:4d}  loss {losses[i]:.5f}")
    print(f"last       loss {losses[-1]:.5f}")
    y, (_, logits, ids, *_) = layer.forward(x)
    print(f"balance    loss {layer.balance_loss(logits, ids)[0].mean().item():.4f} (1 is even)")
    layer.quantise()
    off = (layer.forward_int8(x).float() - y.float()).norm() / y.float().norm()
    print(f"8 bits     {off.item():.4f} from the bf16 layer's outputs")


if __name__ == "__main__":
    main()
