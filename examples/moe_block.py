"""A mixture-of-experts block over two ranks, on one GPU: every operator of the
block as a program calls it. The ranks' experts are two sets of weights here;
with one process per GPU each runs its own part of the loop, and the norm
reads its peers' partial results as it reads the two here.

    python examples/moe_block.py

serve(): one step with 8-bit experts: tokens sorted by expert and quantized on
the way, two products with an activation between, rows back at their tokens,
and the ranks' sum with the norms, the gate and the residual.
train(): the same block in BF16 and its gradient down to the tokens, the
router's weights, the residual stream, the gate and the norms' weights.
Both are compared with plain torch in float64.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allreduce_reduction_rx_amd as rx  # noqa: E402

RANKS, EPS = 2, 1e-5
BF16, FP32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32


def empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Block:
    """Weights and inputs of a block: `experts` experts on each rank."""

    def __init__(self, tokens=96, hidden=256, inner=512, experts=4, topk=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16)
        self.tokens, self.hidden, self.inner, self.experts, self.topk = tokens, hidden, inner, experts, topk
        self.x, self.residual = rnd(tokens, hidden), rnd(tokens, hidden)
        self.gate, self.w_post, self.w_pre = rnd(1, hidden), 1 + rnd(hidden, scale=0.1), 1 + rnd(hidden, scale=0.1)
        self.up = [rnd(experts, inner, hidden, scale=hidden ** -0.5) for _ in range(RANKS)]
        self.down = [rnd(experts, hidden, inner, scale=inner ** -0.5) for _ in range(RANKS)]
        score = torch.randn(tokens, RANKS * experts, generator=g, device="cuda")
        top, ids = torch.topk(score, topk, dim=1)
        self.ids, self.weights = ids.to(I32).contiguous(), torch.softmax(top, dim=1).contiguous()

    def plan_buffers(self):
        pairs = self.tokens * self.topk
        return empty(self.experts + 1, dtype=I32), empty(pairs, dtype=I32), empty(self.tokens, self.topk, dtype=I32)

    def workspace(self):
        n = rx.rx_moe_dispatch_workspace(self.tokens, self.topk, self.experts)
        return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def quantized(w):
    """Weights to int8 with a scale for each channel, once, when they are loaded."""
    e, n, k = w.shape
    codes, scales = empty(e, n, k, dtype=I8), empty(e, n, dtype=FP32)
    rx.rx_quant_i8(w.view(e * n, k), codes.view(e * n, k), scales.view(e * n))
    return codes, scales


def serve(b):
    """h and z of one step, from weights quantized beforehand."""
    up, down = [quantized(w) for w in b.up], [quantized(w) for w in b.down]
    pairs, partial = b.tokens * b.topk, []
    for r in range(RANKS):
        offsets, order, slots = b.plan_buffers()
        codes, scales = empty(pairs, b.hidden, dtype=I8), empty(pairs, dtype=FP32)
        rx.rx_moe_dispatch(b.ids, b.experts, offsets, order, slots, x=b.x, rows=codes, scales=scales,
                           first_expert=r * b.experts, workspace=b.workspace())
        mid = empty(pairs, b.inner)
        rx.rx_gemm_i8(codes, scales, *up[r], mid, offsets=offsets)
        act = F.silu(mid)
        codes, scales = empty(pairs, b.inner, dtype=I8), empty(pairs, dtype=FP32)
        rx.rx_quant_i8(act, codes, scales)
        rows, out = empty(pairs, b.hidden), empty(b.tokens, b.hidden)
        rx.rx_gemm_i8(codes, scales, *down[r], rows, offsets=offsets)
        rx.rx_moe_combine(rows, slots, b.weights, out)
        partial.append(out)
    h, z = empty(b.tokens, b.hidden), empty(b.tokens, b.hidden)
    rx.rx_residual_norm(partial, b.residual, b.gate, b.w_post, b.w_pre, h, z, eps=EPS)
    return h, z


def train(b, d_h, d_z):
    """h and z, and the gradients of (h d_h + z d_z).sum()."""
    pairs, ranks, partial = b.tokens * b.topk, [], []
    for r in range(RANKS):
        offsets, order, slots = b.plan_buffers()
        rows = empty(pairs, b.hidden)
        rx.rx_moe_dispatch(b.ids, b.experts, offsets, order, slots, x=b.x, rows=rows, first_expert=r * b.experts,
                           workspace=b.workspace())
        # the experts' own products are the model's: plain torch here
        rows.requires_grad_()
        ends = offsets.tolist()
        y = torch.cat([F.silu(rows[lo:hi] @ b.up[r][e].t()) @ b.down[r][e].t()
                       for e, (lo, hi) in enumerate(zip(ends, ends[1:]))] + [rows[ends[-1]:] * 0])
        out = empty(b.tokens, b.hidden)
        rx.rx_moe_combine(y.detach(), slots, b.weights, out)
        partial.append(out)
        ranks.append((offsets, slots, rows, y))
    h, z, d_src, d_residual = (empty(b.tokens, b.hidden) for _ in range(4))
    p, q = empty(b.tokens, dtype=FP32), empty(b.tokens, dtype=FP32)
    rx.rx_residual_norm(partial, b.residual, b.gate, b.w_post, b.w_pre, h, z, rstd_post=p, rstd_pre=q, eps=EPS)

    grads = dict(d_gate=empty(1, b.hidden, dtype=FP32), d_w_post=empty(b.hidden, dtype=FP32), d_w_pre=empty(b.hidden, dtype=FP32))
    ws = empty(rx.rx_residual_norm_backward_workspace(b.tokens, b.hidden), dtype=torch.uint8)
    rx.rx_residual_norm_backward(partial, b.residual, b.gate, b.w_post, b.w_pre, p, q, d_h, d_z, d_src, d_residual,
                                 workspace=ws, **grads)
    d_x, d_weights = 0, 0
    for offsets, slots, rows, y in ranks:   # d_src is the gradient of every rank's partial result
        d_y, d_w = empty(pairs, b.hidden), empty(b.tokens, b.topk, dtype=FP32)
        rx.rx_moe_combine_backward(d_src, y.detach(), slots, b.weights, offsets, d_y, d_w)
        d_rows, = torch.autograd.grad(y, rows, d_y)
        back = empty(b.tokens, b.hidden)
        rx.rx_moe_combine(d_rows.contiguous(), slots, None, back)   # the gather's gradient
        d_x, d_weights = d_x + back.float(), d_weights + d_w
    return h, z, dict(grads, d_x=d_x, d_weights=d_weights, d_residual=d_residual)


def plain(b, d_h, d_z):
    """The block and its gradients in float64, every token through its experts."""
    d = lambda t: t.double().requires_grad_()
    x, res, gate, wp, wz, w = (d(t) for t in (b.x, b.residual, b.gate, b.w_post, b.w_pre, b.weights))
    up, down = torch.cat(b.up).double(), torch.cat(b.down).double()
    y = 0
    for j in range(b.topk):
        rows = []
        for t in range(b.tokens):
            e = int(b.ids[t, j])
            rows.append(down[e] @ F.silu(up[e] @ x[t]))
        y = y + torch.stack(rows) * w[:, j:j + 1]
    norm = lambda v: v / (v.square().mean(1, keepdim=True) + EPS).sqrt()
    h = res + gate * norm(y) * wp
    z = norm(h) * wz
    g = torch.autograd.grad((h * d_h.double() + z * d_z.double()).sum(), (x, w, res, gate, wp, wz))
    return h.detach(), z.detach(), dict(zip(("d_x", "d_weights", "d_residual", "d_gate", "d_w_post", "d_w_pre"), g))


def off(got, want):
    """The largest difference over the root mean square of what is wanted."""
    return ((got.double() - want).abs().max() / want.square().mean().sqrt()).item()


def main():
    b = Block()
    d_h, d_z = torch.randn_like(b.x), torch.randn_like(b.x)
    h, z, g = plain(b, d_h, d_z)
    sh, sz = serve(b)
    th, tz, tg = train(b, d_h, d_z)
    report = {"serve h": off(sh, h), "serve z": off(sz, z), "train h": off(th, h), "train z": off(tz, z)}
    report.update({f"train {k}": off(tg[k], g[k]) for k in g})
    for k, v in report.items():
        print(f"{k:18s} off by {v:.4f} of its root mean square")
    return report


if __name__ == "__main__":
    main()
