"""A mixture-of-experts block from the router's logits to the next layer's input,
over two ranks, on one GPU: the router with its losses, experts with 4-bit
weights, and the ranks' sum with bias, dropout, residual and layer norm. The
ranks' experts are two sets of weights here; with one process per GPU each runs
its own part of the loop, and the norm reads its peers' partial results as it
reads the two here.

    python examples/routed_block.py

serve(): one step with 4-bit experts, without dropout.
train(): the same block in BF16 with dropout, and the gradient of its outputs
and of the router's two losses down to the logits, the tokens, the residual
stream, the bias and the norm's weights.
Both are compared with plain torch in float64, serve() with products of the weights
that its codes stand for, so that what is off is the block's, not the quantization's.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allreduce_reduction_rx_amd as rx  # noqa: E402

RANKS, EPS, DROP, GROUP = 2, 1e-5, 0.1, 32
BALANCE, SPREAD = 0.01, 0.001   # what the losses count
BF16, FP32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Block:
    """Weights and inputs of a block: `experts` experts on each rank; every 16th token is padding."""

    def __init__(self, tokens=96, hidden=256, inner=512, experts=4, topk=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16)
        self.tokens, self.hidden, self.inner, self.experts, self.topk = tokens, hidden, inner, experts, topk
        self.x, self.residual, self.logits = rnd(tokens, hidden), rnd(tokens, hidden), rnd(tokens, RANKS * experts)
        self.mask = torch.arange(tokens, device="cuda") % 16 != 15
        self.bias, self.w, self.b = rnd(hidden, scale=0.1), 1 + rnd(hidden, scale=0.1), rnd(hidden, scale=0.1)
        self.up = [rnd(experts, inner, hidden, scale=hidden ** -0.5) for _ in range(RANKS)]
        self.down = [rnd(experts, hidden, inner, scale=inner ** -0.5) for _ in range(RANKS)]
        self.rng = torch.tensor([seed + 1, 0], device="cuda")

    def route(self, training=False):
        """ids and weights of the tokens' experts; for training lse, counts and losses too."""
        ids, weights = empty(self.tokens, self.topk, dtype=I32), empty(self.tokens, self.topk, dtype=FP32)
        more = {}
        if training:
            n = rx.rx_moe_route_workspace(self.tokens, RANKS * self.experts)
            more = dict(lse=empty(self.tokens, dtype=FP32), counts=empty(RANKS * self.experts + 1, dtype=I32), losses=empty(2, dtype=FP32))
            rx.rx_moe_route(self.logits, ids, weights, self.mask, renormalize=True, workspace=empty(n, dtype=U8), **more)
        else:
            rx.rx_moe_route(self.logits, ids, weights, self.mask, renormalize=True)
        return ids, weights, more

    def dispatch(self, rank, ids):
        """A rank's tokens sorted by its experts."""
        pairs = self.tokens * self.topk
        offsets, order, slots = empty(self.experts + 1, dtype=I32), empty(pairs, dtype=I32), empty(self.tokens, self.topk, dtype=I32)
        n = rx.rx_moe_dispatch_workspace(self.tokens, self.topk, self.experts)
        rows = empty(pairs, self.hidden)
        rx.rx_moe_dispatch(ids, self.experts, offsets, order, slots, x=self.x, rows=rows, first_expert=rank * self.experts,
                           workspace=empty(n, dtype=U8) if n else None)
        return offsets, slots, rows


def quantized(w):
    """Weights to 4 bits with a scale for each group, once, when they are loaded."""
    e, n, k = w.shape
    codes, scales = empty(e, n, (k + 31) // 32 * 16, dtype=U8), empty(e, n, -(-k // GROUP), dtype=FP32)
    rx.rx_quant_fp4(w.view(e * n, k), codes.view(e * n, -1)[:, :(k + 1) // 2], scales.view(e * n, -1), GROUP)
    return codes[:, :, :(k + 1) // 2], scales


def values(codes, scales, k):
    """The weights that codes and scales stand for, in float64."""
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :k].long()
    return torch.cat([level, -level])[code] * scales.double().repeat_interleave(GROUP, -1)[..., :k]


def serve(b):
    """h and z of one step, from weights quantized beforehand."""
    up, down = [quantized(w) for w in b.up], [quantized(w) for w in b.down]
    ids, weights, _ = b.route()
    partial = []
    for r in range(RANKS):
        offsets, slots, rows = b.dispatch(r, ids)
        mid = empty(len(rows), b.inner)
        rx.rx_gemm_fp4(rows, *up[r], mid, GROUP, offsets=offsets)
        back, out = empty(len(rows), b.hidden), empty(b.tokens, b.hidden)
        rx.rx_gemm_fp4(F.silu(mid), *down[r], back, GROUP, offsets=offsets)
        rx.rx_moe_combine(back, slots, weights, out)
        partial.append(out)
    h, z = empty(b.tokens, b.hidden), empty(b.tokens, b.hidden)
    rx.rx_layer_norm(partial, b.residual, b.w, b.b, h, z, bias=b.bias, eps=EPS)
    return h, z


def train(b, d_h, d_z):
    """h, z and the losses, and the gradients of (h d_h + z d_z).sum() + BALANCE balance + SPREAD mean of lse^2."""
    ids, weights, router = b.route(training=True)
    ranks, partial = [], []
    for r in range(RANKS):
        offsets, slots, rows = b.dispatch(r, ids)
        # the experts' own products are the model's: plain torch here
        rows.requires_grad_()
        ends = offsets.tolist()
        y = torch.cat([F.silu(rows[lo:hi] @ b.up[r][e].t()) @ b.down[r][e].t()
                       for e, (lo, hi) in enumerate(zip(ends, ends[1:]))] + [rows[ends[-1]:] * 0])
        out = empty(b.tokens, b.hidden)
        rx.rx_moe_combine(y.detach(), slots, weights, out)
        partial.append(out)
        ranks.append((offsets, slots, rows, y))
    h, z, d_src, d_residual = (empty(b.tokens, b.hidden) for _ in range(4))
    mean, rstd = empty(b.tokens, dtype=FP32), empty(b.tokens, dtype=FP32)
    rx.rx_layer_norm(partial, b.residual, b.w, b.b, h, z, bias=b.bias, mean=mean, rstd=rstd, drop=DROP, rng=b.rng, eps=EPS)

    grads = dict(d_bias=empty(b.hidden, dtype=FP32), d_w=empty(b.hidden, dtype=FP32), d_b=empty(b.hidden, dtype=FP32))
    ws = empty(rx.rx_layer_norm_backward_workspace(b.tokens, b.hidden), dtype=U8)
    rx.rx_layer_norm_backward(h, b.w, mean, rstd, d_h, d_z, d_src, d_residual, drop=DROP, rng=b.rng, workspace=ws, **grads)
    d_x, d_weights = 0, 0
    for offsets, slots, rows, y in ranks:   # d_src is the gradient of every rank's partial result
        d_y, d_w = empty(len(rows), b.hidden), empty(b.tokens, b.topk, dtype=FP32)
        rx.rx_moe_combine_backward(d_src, y.detach(), slots, weights, offsets, d_y, d_w)
        d_rows, = torch.autograd.grad(y, rows, d_y)
        back = empty(b.tokens, b.hidden)
        rx.rx_moe_combine(d_rows.contiguous(), slots, None, back)   # the gather's gradient
        d_x, d_weights = d_x + back.float(), d_weights + d_w
    d_logits = empty(b.tokens, RANKS * b.experts)
    rx.rx_moe_route_backward(b.logits, ids, router["lse"], router["counts"], d_weights, torch.tensor([BALANCE, SPREAD], device="cuda"),
                             d_logits, renormalize=True)
    return h, z, router["losses"], dict(grads, d_x=d_x, d_logits=d_logits, d_residual=d_residual)


def kept(b):
    """What dropout multiplies the block's elements with: the operator's own answer to ones."""
    ones, out = torch.ones(b.tokens, b.hidden, dtype=FP32, device="cuda"), empty(b.tokens, b.hidden, dtype=FP32)
    rx.rx_layer_norm([ones], None, None, None, out, None, drop=DROP, rng=b.rng)
    return out.double()


def plain(b, d_h, d_z, mask, up, down):
    """The block, its losses and its gradients in float64, every token through its experts, whose weights are up and down."""
    d = lambda t: t.double().requires_grad_()
    x, logits, res, bias, w, beta = (d(t) for t in (b.x, b.logits, b.residual, b.bias, b.w, b.b))
    live = b.mask.double()
    top, ids = torch.topk(logits, b.topk, dim=1)
    weights = torch.softmax(top, dim=1) * live[:, None]
    y = 0
    for j in range(b.topk):
        rows = [down[int(ids[t, j])] @ F.silu(up[int(ids[t, j])] @ x[t]) for t in range(b.tokens)]
        y = y + torch.stack(rows) * weights[:, j:j + 1]
    h = res + (y + bias) * mask
    z = F.layer_norm(h, (b.hidden,), w, beta, EPS)
    experts, n = RANKS * b.experts, live.sum()
    f = torch.bincount(ids[b.mask].flatten(), minlength=experts) / (n * b.topk)
    balance = experts * (f * (torch.softmax(logits, 1) * live[:, None]).sum(0) / n).sum()
    spread = (torch.logsumexp(logits, 1).square() * live).sum() / n
    g = torch.autograd.grad((h * d_h.double() + z * d_z.double()).sum() + BALANCE * balance + SPREAD * spread, (x, logits, res, bias, w, beta))
    return h.detach(), z.detach(), torch.stack([balance, spread]).detach(), dict(
        zip(("d_x", "d_logits", "d_residual", "d_bias", "d_w", "d_b"), g))


def off(got, want):
    """The largest difference over the root mean square of what is wanted."""
    return ((got.double() - want).abs().max() / want.square().mean().sqrt()).item()


def main():
    b = Block()
    d_h, d_z = torch.randn_like(b.x), torch.randn_like(b.x)
    h, z, _, _ = plain(b, d_h, d_z, 1.0, *(torch.cat([values(*quantized(w), w.shape[-1]) for w in ws]) for ws in (b.up, b.down)))
    sh, sz = serve(b)
    report = {"serve h": off(sh, h), "serve z": off(sz, z)}
    h, z, losses, g = plain(b, d_h, d_z, kept(b), torch.cat(b.up).double(), torch.cat(b.down).double())
    th, tz, tl, tg = train(b, d_h, d_z)
    report.update({"train h": off(th, h), "train z": off(tz, z), "train losses": off(tl, losses)})
    report.update({f"train {k}": off(tg[k], g[k]) for k in g})
    for k, v in report.items():
        print(f"{k:18s} off by {v:.4f} of its root mean square")
    return report


if __name__ == "__main__":
    main()
