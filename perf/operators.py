"""What is measured of the operators around the allreduce of a mixture-of-experts block.

Four operators, in the order in which one rank of a block uses them:

dispatch  tokens sorted by their experts (rx_moe_dispatch)
linear    activations quantized per token to 8-bit integers, times weights with a scale per channel
          (rx_quant_i8 + rx_gemm_i8), dense or one matrix per expert (rx_moe_dispatch + rx_gemm_i8)
combine   the experts' rows back at their tokens with the router's weights, and its gradient
          (rx_moe_combine, rx_moe_combine_backward)
norm      the sum over the ranks' partial results, normed, gated, added to the residual stream, and normed
          for the next block, and its gradient (rx_residual_norm, rx_residual_norm_backward)
"""
import math

import torch

own = False

EPS = 1e-5
RES_SCALE = 0.75
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoding step: 32 sequences, every expert on this rank
        dict(name="dispatch decode", op="dispatch", tokens=32, topk=8, experts=64, world=1, hidden=8192, dtype="bf16"),
        # a ragged batch in FP32, rows that are no whole vectors, a quarter of the experts here
        dict(name="dispatch ragged", op="dispatch", tokens=5003, topk=6, experts=40, world=4, hidden=2501, dtype="fp32"),
        # a prefill or training batch
        dict(name="dispatch prefill", op="dispatch", tokens=16384, topk=8, experts=128, world=1, hidden=4096, dtype="bf16"),
        # the same decoding step's results back at their tokens
        dict(name="combine decode", op="combine", tokens=32, topk=8, experts=64, world=1, hidden=8192, dtype="bf16", train=False),
        # a training step of expert parallelism over two ranks, forward and backward
        dict(name="combine train", op="combine", tokens=16384, topk=8, experts=128, world=2, hidden=4096, dtype="bf16", train=True),
        # one decoding step after a tensor-parallel block over 8 ranks: 32 x 8192, 512 KiB a rank
        dict(name="norm decode", op="norm", rows=32, hidden=8192, sources=8, dtype="bf16", post=True, gate="channel", gate_rows=0, train=False),
        # a training step in FP32 with odd rows and a gate for each sequence of 100 rows
        dict(name="norm ragged train", op="norm", rows=1111, hidden=5001, sources=3, dtype="fp32", post=True, gate="group", gate_rows=100, train=True),
        # a training step over two ranks' partial results at full size
        dict(name="norm train", op="norm", rows=16384, hidden=8192, sources=2, dtype="bf16", post=True, gate="channel", gate_rows=0, train=True),
        # one decoding step's dense product: the weights' bytes are the work
        dict(name="linear decode", op="linear", tokens=32, topk=0, experts=1, world=1, k=8192, n=8192, dtype="bf16"),
        # a ragged batch through experts, half of them here, widths that fill no tile
        dict(name="experts ragged", op="linear", tokens=777, topk=4, experts=24, world=2, k=2056, n=2100, dtype="bf16"),
        # a prefill batch, dense
        dict(name="linear prefill", op="linear", tokens=8192, topk=0, experts=1, world=1, k=8192, n=8192, dtype="bf16"),
        # a prefill batch through 32 experts here
        dict(name="experts prefill", op="linear", tokens=8192, topk=4, experts=32, world=1, k=4096, n=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row's length: whole vectors most of the time, any number otherwise."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.4 else max(lo, w // 64 * 64)


def draw(rng):
    op = rng.choice(("dispatch", "combine", "norm", "linear"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    size = 2 if dtype == "bf16" else 4
    if op in ("dispatch", "combine"):
        topk, world, hidden = rng.randint(1, 8), rng.choice((1, 1, 2, 4, 8)), _width(rng, 64, 8192)
        experts = max(topk, _log(rng, 4, 256))
        tokens = _log(rng, 1, max(1, min(16384, (1 << 30) // (topk * hidden * size))))
        case = dict(op=op, tokens=tokens, topk=topk, experts=experts, world=world, hidden=hidden, dtype=dtype)
        return dict(case, train=rng.random() < 0.5) if op == "combine" else case
    if op == "norm":
        hidden, sources = _width(rng, 64, 16384), rng.randint(1, 8)
        rows = _log(rng, 1, max(1, min(16384, (1 << 29) // (sources * hidden * size))))
        gate = rng.choice(("none", "channel", "group"))
        return dict(op=op, rows=rows, hidden=hidden, sources=sources, dtype=dtype, post=rng.random() < 0.7, gate=gate,
                    gate_rows=_log(rng, 1, rows) if gate == "group" else 0, train=rng.random() < 0.5)
    k, n = _width(rng, 64, 8192), _width(rng, 64, 8192)
    if rng.random() < 0.5:
        return dict(op=op, tokens=_log(rng, 1, 8192), topk=0, experts=1, world=1, k=k, n=n, dtype=dtype)
    topk, world = rng.randint(1, 8), rng.choice((1, 2, 4))
    experts = max(topk, _log(rng, 4, max(4, min(64, (1 << 29) // (k * n)))))
    tokens = _log(rng, 1, max(1, min(8192, 32768 * 4096 // (topk * max(n, k)))))
    return dict(op=op, tokens=tokens, topk=topk, experts=experts, world=world, k=k, n=n, dtype=dtype)


def _first(case):
    """The first expert on this rank, the second rank where there are several."""
    return case["experts"] if case["world"] > 1 else 0


def _routing(case, g):
    """The router's choices: distinct experts a token, some more popular than others, and every 50th
    token padding that goes nowhere. Ids and weights, INT32 and FP32."""
    total = case["experts"] * case["world"]
    t, k = case["tokens"], case["topk"]
    score = torch.randn(t, total, generator=g, device="cuda") + 0.5 * torch.randn(total, generator=g, device="cuda")
    top, ids = torch.topk(score, k, dim=1)
    ids = ids.to(torch.int32)
    ids[49::50] = -1
    return ids.contiguous(), torch.softmax(top, dim=1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(case=dict(case))
    op = case["op"]
    if op == "norm":
        r, h = case["rows"], case["hidden"]
        groups = {"none": 0, "channel": 1, "group": -(-r // max(1, case["gate_rows"]))}[case["gate"]]
        s["gate_rows"] = case["gate_rows"] if case["gate"] == "group" else r
        s["srcs"] = [normal(r, h) for _ in range(case["sources"])]
        s["residual"] = normal(r, h, scale=2.0)
        s["gate"] = normal(groups, h, scale=0.5) if groups else None
        s["w_post"] = (1 + 0.1 * normal(h, dtype=torch.float32)).to(dt) if case["post"] else None
        s["w_pre"] = (1 + 0.1 * normal(h, dtype=torch.float32)).to(dt)
        s["out_h"], s["out_z"] = empty(r, h), empty(r, h)
        s["rstd_post"], s["rstd_pre"] = empty(r, dtype=torch.float32), empty(r, dtype=torch.float32)
        if case["train"]:
            s["d_h"], s["d_z"] = normal(r, h), normal(r, h)
            s["d_src"], s["d_residual"] = empty(r, h), empty(r, h)
            s["d_gate"] = empty(groups, h, dtype=torch.float32) if groups else None
            s["d_w_post"] = empty(h, dtype=torch.float32) if case["post"] else None
            s["d_w_pre"] = empty(h, dtype=torch.float32)
        return s

    if op == "linear":
        t, k, n, e = case["tokens"], case["k"], case["n"], case["experts"]
        pitch = -(-k // 16) * 16
        s["x"] = normal(t, k)
        w = torch.randint(-127, 128, (e, n, pitch), generator=g, device="cuda", dtype=torch.int8)
        s["w"] = w[:, :, :k] if case["topk"] else w[0, :, :k]
        ws = (0.5 + torch.rand(e, n, generator=g, device="cuda")) / (73 * math.sqrt(k))
        s["w_scales"] = ws if case["topk"] else ws[0]
        rows = t * case["topk"] if case["topk"] else t
        s["codes"] = torch.empty(rows, pitch, dtype=torch.int8, device="cuda")[:, :k]
        s["scales"] = empty(rows, dtype=torch.float32)
        s["out"] = empty(rows, n)
        if not case["topk"]:
            return s
    s["ids"], s["weights"] = _routing(case, g)
    t, k, e = case["tokens"], case["topk"], case["experts"]
    i32 = dict(dtype=torch.int32)
    s["offsets"], s["order"], s["slots"] = empty(e + 1, **i32), empty(t * k, **i32), empty(t, k, **i32)
    if op == "dispatch":
        s["x"] = normal(t, case["hidden"])
        s["rows"] = empty(t * k, case["hidden"])
    elif op == "combine":
        h = case["hidden"]
        s["offsets"], s["order"], s["slots"] = _sorted(s["ids"], _first(case), e)
        s["rows"] = normal(t * k, h)
        s["out"] = empty(t, h)
        if case["train"]:
            s["d_out"] = normal(t, h)
            s["d_rows"] = empty(t * k, h)
            s["d_weights"] = empty(t, k, dtype=torch.float32)
    return s


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


# ---- the framework's calls ---------------------------------------------------

def _workspace(s, nbytes):
    """The workspace of a call, kept with the state as a program keeps it."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_dispatch(s):
    import allreduce_reduction_rx_amd as rx

    c = s["case"]
    ws = _workspace(s, lambda: rx.rx_moe_dispatch_workspace(c["tokens"], c["topk"], c["experts"]))
    rx.rx_moe_dispatch(s["ids"], c["experts"], s["offsets"], s["order"], s["slots"], x=s["x"], rows=s["rows"],
                       first_expert=_first(c), workspace=ws)
    return s["offsets"], s["order"], s["slots"], s["rows"]


def _own_combine(s):
    import allreduce_reduction_rx_amd as rx

    rx.rx_moe_combine(s["rows"], s["slots"], s["weights"], s["out"])
    if not s["case"]["train"]:
        return s["out"]
    rx.rx_moe_combine_backward(s["d_out"], s["rows"], s["slots"], s["weights"], s["offsets"], s["d_rows"],
                               s["d_weights"])
    return s["out"], s["d_rows"], s["d_weights"]


def _own_norm(s):
    import allreduce_reduction_rx_amd as rx

    c = s["case"]
    rx.rx_residual_norm(s["srcs"], s["residual"], s["gate"], s["w_post"], s["w_pre"], s["out_h"], s["out_z"],
                        rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], gate_rows=s["gate_rows"],
                        residual_scale=RES_SCALE, eps=EPS)
    if not c["train"]:
        return s["out_h"], s["out_z"]
    ws = _workspace(s, lambda: rx.rx_residual_norm_backward_workspace(c["rows"], c["hidden"], s["gate_rows"]))
    rx.rx_residual_norm_backward(s["srcs"], s["residual"], s["gate"], s["w_post"], s["w_pre"], s["rstd_post"],
                                 s["rstd_pre"], s["d_h"], s["d_z"], s["d_src"], s["d_residual"], d_gate=s["d_gate"],
                                 d_w_post=s["d_w_post"], d_w_pre=s["d_w_pre"], gate_rows=s["gate_rows"],
                                 residual_scale=RES_SCALE, workspace=ws)
    return dict(h=s["out_h"], z=s["out_z"], d_src=s["d_src"], d_residual=s["d_residual"], d_gate=s["d_gate"],
                d_w_post=s["d_w_post"], d_w_pre=s["d_w_pre"])


def _own_linear(s):
    import allreduce_reduction_rx_amd as rx

    c = s["case"]
    if not c["topk"]:
        rx.rx_quant_i8(s["x"], s["codes"], s["scales"])
        rx.rx_gemm_i8(s["codes"], s["scales"], s["w"], s["w_scales"], s["out"])
        return s["scales"], s["out"]
    ws = _workspace(s, lambda: rx.rx_moe_dispatch_workspace(c["tokens"], c["topk"], c["experts"]))
    rx.rx_moe_dispatch(s["ids"], c["experts"], s["offsets"], s["order"], s["slots"], x=s["x"], rows=s["codes"],
                       scales=s["scales"], first_expert=_first(c), workspace=ws)
    rx.rx_gemm_i8(s["codes"], s["scales"], s["w"], s["w_scales"], s["out"], offsets=s["offsets"])
    return s["offsets"], s["slots"], s["scales"], s["out"]


_own = dict(dispatch=_own_dispatch, combine=_own_combine, norm=_own_norm, linear=_own_linear)


# ---- the plain forms -----------------------------------------------------------

def _sorted(ids, first, experts):
    """offsets, order and slots of a stable sort by expert; experts elsewhere come last and have none."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= first) & (flat < first + experts), flat - first, experts)
    order = torch.argsort(key, stable=True)
    ends = torch.searchsorted(key[order], torch.arange(experts, device=key.device), right=True)
    offsets = torch.cat([ends.new_zeros(1), ends])
    place = torch.arange(key.numel(), device=key.device)
    slots = torch.empty_like(place)
    slots[order] = place
    kept = offsets[-1]
    slots = torch.where(slots < kept, slots, -1)
    order = torch.where(place < kept, order, -1)
    return offsets.to(torch.int32), order.to(torch.int32), slots.to(torch.int32).reshape(ids.shape)


def _plain_dispatch(s):
    c = s["case"]
    offsets, order, slots = _sorted(s["ids"], _first(c), c["experts"])
    rows = s["x"][order.clamp(min=0).long() // c["topk"]]
    rows[order < 0] = 0
    return offsets, order, slots, rows


def _plain_combine(s):
    slots = s["slots"].long()
    kept = (slots >= 0)[..., None]
    picked = torch.where(kept, s["rows"][slots.clamp(min=0)].float(), 0.0)
    weights = s["weights"]
    out = (picked * weights[..., None]).sum(1).to(s["rows"].dtype)
    if not s["case"]["train"]:
        return out
    d_out = s["d_out"].float()[:, None]
    d_weights = (picked * d_out).sum(-1)
    d_rows = torch.zeros_like(s["rows"])
    owned = kept[..., 0]
    d_rows[slots[owned]] = (weights[..., None] * d_out).to(d_rows.dtype)[owned]
    return out, d_rows, d_weights


def _plain_norm(s):
    c = s["case"]
    y = sum(t.float() for t in s["srcs"])
    res, w_pre = s["residual"].float(), s["w_pre"].float()
    gate = s["gate"].float() if s["gate"] is not None else None
    row = torch.arange(y.shape[0], device=y.device) // s["gate_rows"]
    g = gate[row] if gate is not None else 1.0
    w_post = s["w_post"].float() if c["post"] else 1.0
    p = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if c["post"] else 1.0
    u = y * p * w_post
    h = RES_SCALE * res + g * u
    q = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    z = h * q * w_pre
    dt = s["residual"].dtype
    if not c["train"]:
        return h.to(dt), z.to(dt)
    d_h, d_z = s["d_h"].float(), s["d_z"].float()
    a = d_z * w_pre
    d_full = d_h + q * (a - h * q * q * (a * h).mean(-1, keepdim=True))
    d_u = d_full * g
    b = d_u * w_post
    d_y = p * (b - y * p * p * (b * y).mean(-1, keepdim=True)) if c["post"] else b
    d_gate = torch.zeros_like(gate).index_add_(0, row, d_full * u) if gate is not None and c["gate"] == "group" else \
        (d_full * u).sum(0, keepdim=True) if gate is not None else None
    return dict(h=h.to(dt), z=z.to(dt), d_src=d_y.to(dt), d_residual=(RES_SCALE * d_full).to(dt), d_gate=d_gate,
                d_w_post=(d_u * y * p).sum(0) if c["post"] else None, d_w_pre=(d_z * h * q).sum(0))


def _quantized(x):
    """8-bit codes (as FP32 values) and a scale for each row; the quotients are taken in 64 bits and rounded once."""
    x = x.float()
    top = x.abs().amax(-1).double()
    scale, inverse = (top / 127).float(), (127 / top).float()
    flat = (top == 0) | (scale == 0) | ~torch.isfinite(inverse)
    scale, inverse = torch.where(flat, 1.0, scale), torch.where(flat, 1.0, inverse)
    return (x * inverse[:, None]).round().clamp(-127, 127), scale


def _plain_linear(s):
    c = s["case"]
    codes, scales = _quantized(s["x"])
    if not c["topk"]:
        total = codes @ s["w"].float().t()
        return scales, (total * scales[:, None] * s["w_scales"]).to(s["x"].dtype)
    offsets, order, slots = _sorted(s["ids"], _first(c), c["experts"])
    kept = order >= 0
    token = order.clamp(min=0).long() // c["topk"]
    scales = torch.where(kept, scales[token], 1.0)
    at = torch.arange(order.numel(), device=order.device)
    expert = torch.searchsorted(offsets[1:].long(), at, right=True).clamp(max=c["experts"] - 1)
    room = max(1, int((offsets[1:] - offsets[:-1]).max()))
    place = expert * room + at - offsets.long()[expert]
    padded = codes.new_zeros(c["experts"] * room, c["k"])
    padded[place[kept]] = codes[token[kept]]
    total = torch.bmm(padded.view(c["experts"], room, c["k"]), s["w"].float().transpose(1, 2).contiguous())
    out = s["out"].new_zeros(order.numel(), c["n"])
    rows = total.view(-1, c["n"])[place[kept]]
    out[kept] = (rows * scales[kept][:, None] * s["w_scales"][expert[kept]]).to(out.dtype)
    return offsets, slots, scales, out


_plain = dict(dispatch=_plain_dispatch, combine=_plain_combine, norm=_plain_norm, linear=_plain_linear)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        r, h, n = case["rows"], case["hidden"], case["sources"]
        groups = {"none": 0, "channel": 1, "group": -(-r // max(1, case["gate_rows"]))}[case["gate"]]
        params = h * (groups + 1 + case["post"])
        if not case["train"]:
            return dict(bytes=e * (r * h * (n + 3) + params), flops=r * h * (n + 10))
        return dict(bytes=e * (r * h * (n + 7) + params) + 4 * params, flops=r * h * (n + 40))
    t, k = case["tokens"], max(1, case["topk"])
    pairs = t * k
    kept = (t - t // 50) * k / case["world"] if case["topk"] else pairs
    plan = 12 * pairs + 4 * case["experts"] if case["topk"] else 0
    if case["op"] == "linear":
        used = case["experts"] * (1 - (1 - 1 / case["experts"]) ** kept) if case["topk"] else 1
        return dict(bytes=e * t * case["k"] + used * case["n"] * (case["k"] + 4) + e * pairs * case["n"] + 4 * pairs + plan,
                    flops=2 * kept * case["k"] * case["n"])
    h = case["hidden"]
    if case["op"] == "dispatch":
        return dict(bytes=e * h * (t + pairs) + plan, flops=0)
    if not case["train"]:
        return dict(bytes=e * h * (t + kept) + 8 * pairs, flops=2 * kept * h)
    return dict(bytes=e * h * (2 * t + kept + pairs) + 12 * pairs, flops=5 * kept * h)


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_plan(ids, first, experts):
    """Offsets, order and slots counted on the host, expert after expert."""
    flat = ids.reshape(-1).cpu() - first
    order = [torch.nonzero(flat == e).reshape(-1) for e in range(experts)]
    offsets = torch.tensor([0] + [o.numel() for o in order]).cumsum(0)
    kept = torch.cat(order)
    full = torch.full((flat.numel(),), -1, dtype=torch.long)
    full[: kept.numel()] = kept
    slots = torch.full((flat.numel(),), -1, dtype=torch.long)
    slots[kept] = torch.arange(kept.numel())
    return offsets, full, slots.reshape(ids.shape)


def _exact_codes(x):
    """fl32(127 / A) and fl32(A / 127) are part of the definition, and so is the product's rounding to 32 bits."""
    x = x.double()
    top = x.abs().max(dim=-1).values
    scale, inverse = (top / 127).float().double(), (127 / top).float().double()
    one = (top == 0) | (scale == 0) | torch.isinf(inverse)
    scale[one], inverse[one] = 1.0, 1.0
    codes = torch.round((x * inverse[:, None]).float()).double()
    return torch.clamp(codes, -127, 127), scale


def _exact_linear(case, s):
    codes, scales = _exact_codes(s["x"])
    if not case["topk"]:
        return scales, (codes * scales[:, None]) @ (s["w"].double() * s["w_scales"].double()[:, None]).t()
    offsets, order, slots = _exact_plan(s["ids"], _first(case), case["experts"])
    n_kept = int(offsets[-1])
    token = (order[:n_kept] // case["topk"]).cuda()
    all_scales = torch.ones(order.numel(), dtype=torch.float64, device="cuda")
    all_scales[:n_kept] = scales[token]
    out = torch.zeros(order.numel(), case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            t = token[lo:hi]
            out[lo:hi] = (codes[t] @ s["w"][e].double().t()) * scales[t][:, None] * s["w_scales"][e].double()
    return offsets.int(), slots.int(), all_scales, out


def _exact_norm(case, s):
    d = {k: (v.double() if torch.is_tensor(v) else v) for k, v in s.items()}
    y = torch.stack([t.double() for t in s["srcs"]]).sum(0)
    hidden = y.shape[1]
    groups = torch.arange(y.shape[0], device="cuda").div(s["gate_rows"], rounding_mode="floor")
    g = d["gate"].index_select(0, groups) if s["gate"] is not None else torch.ones_like(y)
    if case["post"]:
        norm = (y.square().sum(1, keepdim=True) / hidden + EPS).sqrt()
        unit = y / norm
        u = unit * d["w_post"]
    else:
        u = y
    h = d["residual"] * RES_SCALE + g * u
    norm_h = (h.square().sum(1, keepdim=True) / hidden + EPS).sqrt()
    unit_h = h / norm_h
    z = unit_h * d["w_pre"]
    if not case["train"]:
        return h, z
    through = d["d_z"] * d["w_pre"]
    full = d["d_h"] + (through - unit_h * (through * unit_h).sum(1, keepdim=True) / hidden) / norm_h
    back = full * g
    d_gate = None
    if s["gate"] is not None:
        d_gate = torch.zeros_like(d["gate"]).index_add(0, groups, full * u)
    if case["post"]:
        d_w_post = (back * unit).sum(0)
        into = back * d["w_post"]
        d_src = (into - unit * (into * unit).sum(1, keepdim=True) / hidden) / norm
    else:
        d_w_post, d_src = None, back
    return dict(h=h, z=z, d_src=d_src, d_residual=full * RES_SCALE, d_gate=d_gate, d_w_post=d_w_post,
                d_w_pre=(d["d_z"] * unit_h).sum(0))


def _exact_combine(case, s):
    t, k = case["tokens"], case["topk"]
    slots = s["slots"].long()
    h = case["hidden"]
    out = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    d_rows = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
    d_weights = torch.zeros(t, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        here = torch.nonzero(slots[:, j] >= 0).reshape(-1)
        at, w = slots[here, j], s["weights"][here, j].double()[:, None]
        rows = s["rows"][at].double()
        out[here] += w * rows
        if case["train"]:
            grad = s["d_out"][here].double()
            d_rows[at] = w * grad
            d_weights[here, j] = (rows * grad).sum(1)
    return (out, d_rows, d_weights) if case["train"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(case, s)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "combine":
        return _exact_combine(case, s)
    offsets, order, slots = _exact_plan(s["ids"], _first(case), case["experts"])
    rows = torch.zeros(order.numel(), case["hidden"], dtype=torch.float64, device="cuda")
    kept = order >= 0
    rows[kept.cuda()] = s["x"].double()[(order[kept] // case["topk"]).cuda()]
    return offsets.int(), order.int(), slots.int(), rows
