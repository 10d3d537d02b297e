"""What is measured of the operators before and behind the experts of a mixture-of-experts block, and of
blocks whose weights are held in 4 bits or whose end is a layer norm with dropout.

Three operators, in the order in which one rank of a block uses them:

route      each token's experts from the router's logits, their weights, the counts and the two losses of the
           router, and the gradient of all of it (rx_moe_route, rx_moe_route_backward)
linear4    rows of activations times weights of 4 bits with a scale for each group, dense or one matrix per
           expert (rx_gemm_fp4)
layernorm  the sum over the ranks' partial results with bias, dropout, residual and layer norm, and its
           gradient (rx_layer_norm, rx_layer_norm_backward)
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # magnitudes of E2M1; bit 3 is the sign


def listed():
    return [
        # one decoding step: 32 sequences
        dict(name="route decode", op="route", tokens=32, experts=64, topk=8, dtype="bf16", renormalize=False, closed=0, train=False),
        # a ragged batch in FP32, experts that are no power of two, some of them on a rank that is gone
        dict(name="route ragged train", op="route", tokens=5003, experts=160, topk=6, dtype="fp32", renormalize=True, closed=20, train=True),
        # a training batch
        dict(name="route train", op="route", tokens=16384, experts=128, topk=8, dtype="bf16", renormalize=False, closed=0, train=True),
        # one sequence's decoding step through a dense product: the weights' bytes are the work
        dict(name="linear4 single", op="linear4", tokens=1, topk=0, experts=1, world=1, k=8192, n=8192, group=128, dtype="bf16"),
        # the same for 32 sequences, a scale for each 32 weights
        dict(name="linear4 decode", op="linear4", tokens=32, topk=0, experts=1, world=1, k=8192, n=8192, group=32, dtype="bf16"),
        # 32 sequences' decoding step through 64 experts
        dict(name="experts4 decode", op="linear4", tokens=32, topk=8, experts=64, world=1, k=4096, n=4096, group=128, dtype="bf16"),
        # a ragged batch in FP32 through experts, half of them here, widths that fill no tile and no group
        dict(name="experts4 ragged", op="linear4", tokens=777, topk=4, experts=24, world=2, k=2056, n=2100, group=64, dtype="fp32"),
        # a short prompt, dense
        dict(name="linear4 prefill", op="linear4", tokens=1024, topk=0, experts=1, world=1, k=8192, n=8192, group=128, dtype="bf16"),
        # one decoding step after a tensor-parallel block over 8 ranks
        dict(name="layernorm decode", op="layernorm", rows=32, hidden=8192, sources=8, dtype="bf16", residual=True, bias=True, drop=0.0, train=False),
        # a training step in FP32 with odd rows
        dict(name="layernorm ragged train", op="layernorm", rows=1111, hidden=5001, sources=3, dtype="fp32", residual=True, bias=True, drop=0.1, train=True),
        # the norm before a block: one source, nothing to add
        dict(name="layernorm alone train", op="layernorm", rows=8192, hidden=4096, sources=1, dtype="bf16", residual=False, bias=False, drop=0.0, train=True),
        # a training step over two ranks' partial results at full size
        dict(name="layernorm train", op="layernorm", rows=16384, hidden=8192, sources=2, dtype="bf16", residual=True, bias=True, drop=0.1, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row's length: whole vectors most of the time, any number otherwise."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.4 else max(lo, w // 64 * 64)


def draw(rng):
    op = rng.choice(("route", "linear4", "linear4", "layernorm"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    size = 2 if dtype == "bf16" else 4
    if op == "route":
        experts = _log(rng, 4, 512)
        return dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, topk=rng.randint(1, min(16, experts)), dtype=dtype,
                    renormalize=rng.random() < 0.5, closed=rng.randint(1, experts - 1) if rng.random() < 0.25 else 0,
                    train=rng.random() < 0.6)
    if op == "layernorm":
        hidden, sources = _width(rng, 64, 16384), rng.randint(1, 8)
        rows = _log(rng, 1, max(1, min(16384, (1 << 29) // (sources * hidden * size))))
        return dict(op=op, rows=rows, hidden=hidden, sources=sources, dtype=dtype, residual=rng.random() < 0.7,
                    bias=rng.random() < 0.5, drop=rng.choice((0.0, 0.1, 0.3)), train=rng.random() < 0.5)
    k, n, group = _width(rng, 64, 8192), _width(rng, 64, 8192), rng.choice((32, 64, 128))
    if rng.random() < 0.5:
        return dict(op=op, tokens=_log(rng, 1, 1024), topk=0, experts=1, world=1, k=k, n=n, group=group, dtype=dtype)
    topk, world = rng.randint(1, 8), rng.choice((1, 2, 4))
    experts = max(topk, _log(rng, 4, max(4, min(64, (1 << 29) // (k * n)))))
    tokens = _log(rng, 1, max(1, min(1024, 4096 * 4096 // (topk * max(n, k)))))
    return dict(op=op, tokens=tokens, topk=topk, experts=experts, world=world, k=k, n=n, group=group, dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)

    def normal(*shape, dtype=dt, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(case=dict(case))
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        # some experts more popular than others, every 50th token padding, the last experts closed
        logits = normal(t, e, dtype=torch.float32, scale=1.5) + normal(1, e, dtype=torch.float32, scale=0.7)
        if case["closed"]:
            logits[:, e - case["closed"]:] = -math.inf
        s["logits"] = logits.to(dt)
        s["mask"] = torch.ones(t, dtype=torch.bool, device="cuda")
        s["mask"][49::50] = False
        s["ids"], s["weights"], s["lse"] = empty(t, k, **i32), empty(t, k, **f32), empty(t, **f32)
        s["counts"], s["losses"] = empty(e + 1, **i32), empty(2, **f32)
        if case["train"]:
            s["d_weights"] = normal(t, k, **f32)
            # what the losses' coefficients make of them, and a gradient of about one for each token
            s["d_losses"] = torch.tensor([0.5 * t, 0.1 * t], device="cuda") * (0.5 + torch.rand(2, generator=g, device="cuda"))
            s["d_logits"] = empty(t, e)
        return s

    if op == "layernorm":
        r, h = case["rows"], case["hidden"]
        s["srcs"] = [normal(r, h) for _ in range(case["sources"])]
        s["residual"] = normal(r, h, scale=2.0, mean=0.5) if case["residual"] else None
        s["bias"] = normal(h, scale=0.5) if case["bias"] else None
        s["w"], s["b"] = normal(h, scale=0.1, mean=1.0), normal(h, scale=0.1)
        # seed and offset of the generator
        s["rng"] = torch.randint(-(1 << 62), 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64) if case["drop"] else None
        alone = case["sources"] == 1 and not (case["residual"] or case["bias"] or case["drop"])
        s["out_h"], s["out_z"] = None if alone else empty(r, h), empty(r, h)
        s["mean"], s["rstd"] = empty(r, **f32), empty(r, **f32)
        if case["train"]:
            s["d_h"], s["d_z"] = normal(r, h), normal(r, h)
            s["d_src"], s["d_residual"] = empty(r, h), empty(r, h) if case["residual"] else None
            s["d_bias"] = empty(h, **f32) if case["bias"] else None
            s["d_w"], s["d_b"] = empty(h, **f32), empty(h, **f32)
        return s

    t, k, n, e = case["tokens"], case["k"], case["n"], case["experts"]
    half, pitch, groups = -(-k // 2), -(-k // 32) * 16, -(-k // case["group"])
    codes = torch.randint(0, 256, (e, n, pitch), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.5 + torch.rand(e, n, groups, generator=g, device="cuda")) / (3 * math.sqrt(k))
    s["codes"], s["scales"] = codes[:, :, :half], scales
    if not case["topk"]:
        s["codes"], s["scales"] = s["codes"][0], scales[0]
        s["x"], s["out"] = normal(t, k), empty(t, n)
        return s
    # the plan of a dispatch: distinct experts a token, some more popular, the first rank of several
    total = e * case["world"]
    score = torch.randn(t, total, generator=g, device="cuda") + 0.5 * torch.randn(total, generator=g, device="cuda")
    ids = torch.topk(score, case["topk"], dim=1)[1].reshape(-1)
    count = torch.bincount(ids, minlength=total)[:e]
    s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    rows = t * case["topk"]
    s["x"], s["out"] = normal(rows, k), empty(rows, n)
    return s


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


# ---- the framework's calls ---------------------------------------------------

def _workspace(s, nbytes):
    """The workspace of a call, kept with the state as a program keeps it."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_route(s):
    import allreduce_reduction_rx_amd as rx

    c = s["case"]
    ws = _workspace(s, lambda: rx.rx_moe_route_workspace(c["tokens"], c["experts"]))
    rx.rx_moe_route(s["logits"], s["ids"], s["weights"], token_mask=s["mask"], renormalize=c["renormalize"], lse=s["lse"],
                    counts=s["counts"], losses=s["losses"], workspace=ws)
    out = dict(ids=s["ids"], weights=s["weights"], lse=s["lse"], counts=s["counts"], losses=s["losses"])
    if c["train"]:
        rx.rx_moe_route_backward(s["logits"], s["ids"], s["lse"], s["counts"], s["d_weights"], s["d_losses"], s["d_logits"],
                                 renormalize=c["renormalize"])
        out["d_logits"] = s["d_logits"]
    return out


def _own_linear4(s):
    import allreduce_reduction_rx_amd as rx

    rx.rx_gemm_fp4(s["x"], s["codes"], s["scales"], s["out"], s["case"]["group"], offsets=s.get("offsets"))
    return s["out"]


def _own_layernorm(s):
    import allreduce_reduction_rx_amd as rx

    c = s["case"]
    rx.rx_layer_norm(s["srcs"], s["residual"], s["w"], s["b"], s["out_h"], s["out_z"], bias=s["bias"], mean=s["mean"],
                     rstd=s["rstd"], drop=c["drop"], rng=s["rng"], eps=EPS)
    out = dict(h=s["out_h"], z=s["out_z"], mean=s["mean"], rstd=s["rstd"])
    if c["train"]:
        ws = _workspace(s, lambda: rx.rx_layer_norm_backward_workspace(c["rows"], c["hidden"]))
        h = s["srcs"][0] if s["out_h"] is None else s["out_h"]
        rx.rx_layer_norm_backward(h, s["w"], s["mean"], s["rstd"], s["d_h"], s["d_z"], s["d_src"], d_residual=s["d_residual"],
                                  d_bias=s["d_bias"], d_w=s["d_w"], d_b=s["d_b"], drop=c["drop"], rng=s["rng"], workspace=ws)
        out.update(d_src=s["d_src"], d_residual=s["d_residual"], d_bias=s["d_bias"], d_w=s["d_w"], d_b=s["d_b"])
    return out


_own = dict(route=_own_route, linear4=_own_linear4, layernorm=_own_layernorm)


# ---- the plain forms -----------------------------------------------------------

def _plain_route(s):
    c = s["case"]
    e, k = c["experts"], c["topk"]
    x = s["logits"].float()
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = value[:, :k], order[:, :k]
    live = s["mask"] & (value[:, 0] > -math.inf)
    high = torch.where(live, value[:, 0], 0.0)[:, None]
    raised = torch.where(live[:, None], (x - high).exp(), 0.0)
    total = torch.where(live, raised.sum(1), 1.0)[:, None]
    prob = raised / total
    lse = torch.where(live, high[:, 0] + total[:, 0].log(), -math.inf)
    kept = live[:, None] & (top > -math.inf)
    chosen = torch.where(kept, (top - high).exp(), 0.0)
    share = torch.where(live, chosen.sum(1), 1.0)[:, None]
    weights = chosen / (share if c["renormalize"] else total)
    tokens = live.sum()
    counts = torch.cat([torch.bincount(ids[kept], minlength=e), tokens[None]])
    n = tokens.clamp(min=1).float()
    rate = counts[:e].float() / (n * k)
    balance = e * (rate * (prob.sum(0) / n)).sum()
    z = torch.where(live, lse.square(), 0.0).sum() / n
    out = dict(ids=torch.where(kept, ids, -1).to(torch.int32), weights=weights, lse=lse, counts=counts.to(torch.int32),
               losses=torch.stack([balance, z]))
    if not c["train"]:
        return out
    g, d = torch.where(kept, s["d_weights"], 0.0), s["d_losses"]
    d_prob = (d[0] * e / n) * rate + torch.zeros_like(prob)
    if c["renormalize"]:
        mean = (weights * g).sum(1, keepdim=True)
        extra = torch.where(kept, weights * (g - mean), 0.0)
    else:
        d_prob = d_prob.scatter_add(1, ids, g)
        extra = torch.zeros_like(g)
    d_logits = prob * (d_prob - (prob * d_prob).sum(1, keepdim=True))
    d_logits = d_logits + torch.where(live, 2 * d[1] / n * lse, 0.0)[:, None] * prob
    d_logits = d_logits.scatter_add(1, ids, extra)
    out["d_logits"] = torch.where(live[:, None], d_logits, 0.0).to(s["logits"].dtype)
    return out


def _weights(codes, scales, k, group):
    """The weights that codes of two a byte (the even one in the low half) and their groups' scales stand for."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :k]
    value = level.index_select(0, pair.reshape(-1).int()).view(pair.shape)
    return value * scales.repeat_interleave(group, dim=-1)[..., :k]


def _plain_linear4(s):
    c = s["case"]
    w = _weights(s["codes"], s["scales"], c["k"], c["group"])
    x = s["x"].float()
    if not c["topk"]:
        return (x @ w.t()).to(s["x"].dtype)
    ends, rows = s["offsets"].long(), x.shape[0]
    at = torch.arange(rows, device=x.device)
    expert = torch.searchsorted(ends[1:], at, right=True)
    kept = expert < c["experts"]
    expert = expert.clamp(max=c["experts"] - 1)
    room = max(1, int((ends[1:] - ends[:-1]).max()))
    place = (expert * room + at - ends[expert])[kept]
    padded = x.new_zeros(c["experts"] * room, c["k"])
    padded[place] = x[kept]
    total = torch.bmm(padded.view(c["experts"], room, c["k"]), w.transpose(1, 2).contiguous())
    out = torch.zeros_like(s["out"])
    out[kept] = total.view(-1, c["n"])[place].to(out.dtype)
    return out


M32 = 0xFFFFFFFF


def _generator(rng, count):
    """`count` times eight numbers of 16 bits: Philox of four words and ten rounds (Salmon and others, 2011) of the
    numbers from zero with the offset above them, keyed with the seed."""
    i = torch.arange(count, device="cuda")
    seed, offset = rng[0], rng[1]
    c0, c1, c2, c3 = i & M32, i >> 32, (offset & M32).expand(count), (offset >> 32 & M32).expand(count)
    k0, k1 = seed & M32, seed >> 32 & M32
    for _ in range(10):
        # products modulo 2^64: their halves are right whatever the sign that the type gives them
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (q >> 32 & M32) ^ c1 ^ k0, q & M32, (p >> 32 & M32) ^ c3 ^ k1, p & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack([c0, c1, c2, c3], 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(count, 8)


def _kept(c, rng):
    """Which elements dropout keeps, eight to a number of the generator, each row from a new one."""
    r, h = c["rows"], c["hidden"]
    per = -(-h // 8)
    return (_generator(rng, r * per).view(r, per * 8) >= round(c["drop"] * 65536))[:, :h]


def _plain_layernorm(s):
    c = s["case"]
    dt, h = s["srcs"][0].dtype, c["hidden"]
    y = s["srcs"][0].float()
    for t in s["srcs"][1:]:
        y = y + t.float()
    if c["bias"]:
        y = y + s["bias"].float()
    kept, gain = None, 1.0
    if c["drop"]:
        kept, gain = _kept(c, s["rng"]), 65536 / (65536 - round(c["drop"] * 65536))
        y = torch.where(kept, y * gain, 0.0)
    if c["residual"]:
        y = s["residual"].float() + y
    h = y.to(dt)
    x, w = h.float(), s["w"].float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = torch.rsqrt(centred.square().mean(1) + EPS)
    unit = centred * rstd[:, None]
    out = dict(h=None if s["out_h"] is None else h, z=(unit * w + s["b"].float()).to(dt), mean=mean, rstd=rstd)
    if not c["train"]:
        return out
    d_z = s["d_z"].float()
    a = d_z * w
    full = s["d_h"].float() + rstd[:, None] * (a - a.mean(1, keepdim=True) - unit * (a * unit).mean(1, keepdim=True))
    d_src = torch.where(kept, full * gain, 0.0) if c["drop"] else full
    return dict(out, d_src=d_src.to(dt), d_residual=full.to(dt) if c["residual"] else None,
                d_bias=d_src.sum(0) if c["bias"] else None, d_w=(d_z * unit).sum(0), d_b=d_z.sum(0))


_plain = dict(route=_plain_route, linear4=_plain_linear4, layernorm=_plain_layernorm)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        t, n, k = case["tokens"], case["experts"], case["topk"]
        once = t * (n * e + 8 * k + 5) + 4 * n
        return dict(bytes=once + (t * (n * e + 4 * k) if case["train"] else 0), flops=t * n * (16 if case["train"] else 6))
    if case["op"] == "layernorm":
        r, h, n = case["rows"], case["hidden"], case["sources"]
        alone = n == 1 and not (case["residual"] or case["bias"] or case["drop"])
        params = h * (2 + case["bias"])
        once = e * (r * h * (n + case["residual"] + 2 - alone) + params) + 8 * r
        if not case["train"]:
            return dict(bytes=once, flops=r * h * (n + 10))
        return dict(bytes=once + e * r * h * (3 + case["residual"]) + 4 * params, flops=r * h * (n + 30))
    t, k, n = case["tokens"], case["k"], case["n"]
    rows = t * max(1, case["topk"])
    kept = rows / case["world"]
    used = case["experts"] * (1 - (1 - 1 / case["experts"]) ** kept) if case["topk"] else 1
    weights = used * n * (k / 2 + 4 * -(-k // case["group"]))
    return dict(bytes=weights + e * (kept * k + rows * n), flops=2 * kept * k * n)


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_route(case, s):
    e, k = case["experts"], case["topk"]
    logits = s["logits"].double()
    live = s["mask"] & ~torch.isinf(logits).all(1)
    at = torch.nonzero(live).reshape(-1)
    x = logits[at].requires_grad_(case["train"])
    number = torch.arange(e, device="cuda").expand(at.numel(), e)
    left, ids = x.detach().clone(), torch.full((at.numel(), k), -1, device="cuda")
    for j in range(k):
        # the largest that is left, the first of equals
        top = left.max(1, keepdim=True).values
        first = torch.where(left == top, number, e).min(1).values
        ids[:, j] = torch.where(torch.isinf(top[:, 0]), -1, first)
        left.scatter_(1, first[:, None], -math.inf)
    soft = torch.softmax(x, 1)
    lse = torch.logsumexp(x, 1)
    taken = ids >= 0
    weights = soft.gather(1, ids.clamp(min=0)) * taken
    if case["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    counts = torch.zeros(e + 1, dtype=torch.long, device="cuda")
    counts.index_add_(0, ids[taken], torch.ones_like(ids[taken]))
    counts[e] = at.numel()
    n = max(1, at.numel())
    losses = torch.stack([e * (counts[:e] / (n * k) * soft.sum(0) / n).sum(), lse.square().sum() / n])

    def whole(v, fill):
        full = torch.full((case["tokens"], *v.shape[1:]), fill, dtype=v.dtype, device="cuda")
        full[at] = v.detach()
        return full

    out = dict(ids=whole(ids, -1).int(), weights=whole(weights, 0), lse=whole(lse, -math.inf), counts=counts.int(),
               losses=losses.detach())
    if case["train"]:
        (weights * s["d_weights"][at].double()).sum().add((losses * s["d_losses"].double()).sum()).backward()
        out["d_logits"] = whole(x.grad, 0)
    return out


def _exact_linear4(case, s):
    k, n, group = case["k"], case["n"], case["group"]
    level = torch.tensor([*LEVELS, *[-v for v in LEVELS]], dtype=torch.float64, device="cuda")

    def product(x, codes, scales):
        w = torch.empty(n, 2 * codes.shape[1], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = level[(codes % 16).long()], level[(codes // 16).long()]
        out = torch.zeros(x.shape[0], n, dtype=torch.float64, device="cuda")
        for i in range(scales.shape[1]):
            lo, hi = i * group, min(k, (i + 1) * group)
            out += (x[:, lo:hi].double() @ w[:, lo:hi].t()) * scales[:, i].double()
        return out

    if not case["topk"]:
        return product(s["x"], s["codes"], s["scales"])
    out = torch.zeros(s["x"].shape[0], n, dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            out[lo:hi] = product(s["x"][lo:hi], s["codes"][e], s["scales"][e])
    return out


def _exact_kept(case, rng):
    """The generator once more, on the host and in unsigned numbers."""
    import numpy as np

    def u32(v):
        return np.uint64(v & M32)

    seed, offset = rng.tolist()
    r, h = case["rows"], case["hidden"]
    per = (h + 7) // 8
    low = np.uint64(M32)
    a = np.arange(r * per, dtype=np.uint64)
    b, a = a >> np.uint64(32), a & low
    c, d = np.full_like(a, u32(offset)), np.full_like(a, u32(offset >> 32))
    keys = [(u32(seed + i * 0x9E3779B9), u32((seed >> 32) + i * 0xBB67AE85)) for i in range(10)]
    for k0, k1 in keys:
        m = a * np.uint64(0xD2511F53)
        a = c * np.uint64(0xCD9E8D57)
        c = (m >> np.uint64(32)) ^ d ^ k1
        d = m & low
        a, b = (a >> np.uint64(32)) ^ b ^ k0, a & low
    half = np.empty((r * per, 8), dtype=np.uint16)
    for j, word in enumerate((a, b, c, d)):
        half[:, 2 * j] = word & np.uint64(0xFFFF)
        half[:, 2 * j + 1] = word >> np.uint64(16)
    kept = half.reshape(r, per * 8)[:, :h] >= round(case["drop"] * 65536)
    return torch.from_numpy(kept).cuda()


def _exact_layernorm(case, s):
    y = torch.stack([t.double() for t in s["srcs"]]).sum(0)
    if case["bias"]:
        y = y + s["bias"].double()
    keep = None
    if case["drop"]:
        drop = round(case["drop"] * 65536) / 65536
        keep = _exact_kept(case, s["rng"]).double() / (1 - drop)
        y = y * keep
    if case["residual"]:
        y = y + s["residual"].double()
    x = y.to(s["srcs"][0].dtype).double()   # the norm is that of h as it is stored
    w, b = s["w"].double(), s["b"].double()
    if case["train"]:
        x.requires_grad_()
        w.requires_grad_()
        b.requires_grad_()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    root = (var + EPS).sqrt()
    z = (x - mean) / root * w + b
    out = dict(h=None if s["out_h"] is None else x.detach(), z=z.detach(), mean=mean.detach()[:, 0], rstd=1 / root.detach()[:, 0])
    if not case["train"]:
        return out
    d_x, d_w, d_b = torch.autograd.grad(z, (x, w, b), s["d_z"].double())
    d_x = d_x + s["d_h"].double()
    d_src = d_x if keep is None else d_x * keep
    return dict(out, d_src=d_src, d_residual=d_x if case["residual"] else None,
                d_bias=d_src.sum(0) if case["bias"] else None, d_w=d_w, d_b=d_b)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, linear4=_exact_linear4, layernorm=_exact_layernorm)[case["op"]](case, s)
