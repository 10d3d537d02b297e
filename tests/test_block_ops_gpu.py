"""The operators around a block's allreduce on the GPU against their float64
forms (block_ref.py, whose bounds are counted from the roundings)."""
import pytest
import torch

import allreduce_reduction_rx_amd as rx
import block_ref as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = [BF16, FP32]


def gpu(t):
    return None if t is None else t.cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=FP32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


class Strided:
    """A rows x width GPU matrix with `extra` guard elements behind every row
    and a guard row on both sides; starts `shift` elements into its storage."""

    def __init__(self, rows, width, dtype, extra=5, shift=1):
        self.ld = width + extra
        self.full = torch.full(((rows + 2) * self.ld + shift,), 77.0 if dtype != torch.int8 else 77, dtype=dtype,
                               device="cuda")
        self.t = torch.as_strided(self.full, (rows, width), (self.ld, 1), shift + self.ld)

    def check(self):
        inside = torch.zeros_like(self.full, dtype=torch.bool)
        torch.as_strided(inside, self.t.shape, self.t.stride(), self.t.storage_offset())[:] = True
        assert bool((self.full[~inside] == 77).all()), "written outside the rows"


def put(m, t):
    m.t.copy_(t)
    return m.t


def within(got, want, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, f"off by {(got - want).abs().max().item():.3g}, {int((over > 0).sum())} values over their bound"


def routing(g, tokens, topk, total, drop=0.0):
    ids = torch.stack([torch.randperm(total, generator=g)[:topk] for _ in range(tokens)]).to(torch.int32) \
        if tokens else torch.zeros(0, topk, dtype=torch.int32)
    if drop:
        ids[torch.rand(tokens, topk, generator=g) < drop] = -1
    return ids


def run_dispatch(ids, experts, first=0, x=None, int8=False, strided=False, stream=None):
    tokens, topk = ids.shape
    pairs = tokens * topk
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, order, slots = (torch.full(s, -77, **i32) for s in ((experts + 1,), (pairs,), (tokens, topk)))
    nbytes = rx.rx_moe_dispatch_workspace(tokens, topk, experts)
    ws = torch.full((nbytes,), 0xA5, dtype=torch.uint8, device="cuda") if nbytes else None
    rows = scales = guard = xg = None
    if x is not None:
        dt = torch.int8 if int8 else x.dtype
        if strided:
            guard = Strided(pairs, x.shape[1], dt)
            rows = guard.t
            xg = put(Strided(tokens, x.shape[1], x.dtype, extra=3), x)
        else:
            rows = torch.full((pairs, x.shape[1]), 77, dtype=dt, device="cuda")
            xg = x.cuda()
        scales = torch.full((pairs,), 77.0, device="cuda") if int8 else None
    idg = ids.cuda()
    rx.rx_moe_dispatch(idg, experts, offsets, order, slots, x=xg, rows=rows, scales=scales, first_expert=first,
                       workspace=ws, stream=stream)
    torch.cuda.synchronize()
    if guard:
        guard.check()
    return offsets.cpu(), order.cpu(), slots.cpu(), None if rows is None else rows.cpu(), \
        None if scales is None else scales.cpu()


# ---- dispatch ------------------------------------------------------------------

PLANS = [  # tokens, topk, experts here, experts in all, first, share of pairs that go nowhere
    (1, 1, 1, 1, 0, 0.0), (1, 8, 8, 64, 3, 0.0), (3, 2, 5, 5, 0, 0.4), (7, 1, 1024, 1024, 0, 0.0),
    (33, 9, 17, 40, 20, 0.1), (5, 64, 100, 100, 0, 0.2), (512, 8, 64, 64, 0, 0.0), (513, 8, 64, 64, 0, 0.02),
    (700, 6, 16, 128, 112, 0.0), (4097, 1, 3, 3, 0, 0.3), (1500, 7, 200, 256, 10, 0.05), (64, 4, 8, 16, 8, 1.0),
    (2000, 3, 4, 8, 4, 1.0), (40000, 8, 8, 8, 0, 0.0),
]


@pytest.mark.parametrize("tokens,topk,experts,total,first,drop", PLANS)
def test_dispatch_plan(tokens, topk, experts, total, first, drop):
    ids = routing(gen(tokens), tokens, topk, total, drop)
    offsets, order, slots, _, _ = run_dispatch(ids, experts, first)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= first) & (flat < first + experts), flat - first, experts)
    by = torch.argsort(key, stable=True)
    kept = int((key < experts).sum())
    assert offsets.tolist() == [int((key < e).sum()) for e in range(experts)] + [kept]
    assert torch.equal(order[:kept].long(), by[:kept]) and bool((order[kept:] == -1).all())
    want = torch.full((tokens * topk,), -1, dtype=torch.int32)
    want[by[:kept]] = torch.arange(kept, dtype=torch.int32)
    assert torch.equal(slots.reshape(-1), want)
    if tokens <= 64:
        for got, ref in zip((offsets, order, slots), R.plan(ids, first, experts)):
            assert torch.equal(got, ref)


def test_dispatch_same_expert_twice_and_extreme_ids():
    ids = torch.tensor([[2, 2, 2], [2 ** 31 - 1, -2 ** 31, 0], [0, 2, 1]], dtype=torch.int32)
    for got, ref in zip(run_dispatch(ids, 3), R.plan(ids, 0, 3)):
        assert torch.equal(got, ref)


def test_dispatch_no_tokens():
    offsets, order, slots, rows, _ = run_dispatch(torch.zeros(0, 2, dtype=torch.int32), 9, x=torch.zeros(0, 8))
    assert offsets.tolist() == [0] * 10 and rows.shape == (0, 8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("tokens,topk,hidden,drop", [
    (1, 1, 1, 0.0), (1, 8, 8192, 0.0), (3, 2, 7, 0.3), (32, 8, 264, 0.1), (9, 12, 1001, 0.1), (600, 8, 130, 0.5),
    (5, 3, 20003, 0.2), (64, 2, 4096, 1.0)])
def test_dispatch_rows(dtype, strided, tokens, topk, hidden, drop):
    g = gen(hidden)
    ids = routing(g, tokens, topk, 16 if topk < 16 else 64, drop)
    x = randn(g, tokens, hidden, dtype=dtype)
    _, order, _, rows, _ = run_dispatch(ids, 12, 0, x, strided=strided)
    assert torch.equal(rows, R.gather(x, order, topk))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("tokens,topk,hidden,experts,total", [
    (4099, 1, 65, 3, 4), (1025, 8, 1000, 100, 256), (70, 60, 2500, 200, 300), (3000, 5, 264, 1024, 1500),
    (4097, 8, 40, 300, 400), (33000, 1, 24, 1000, 1000), (5461, 6, 24, 77, 90)])
def test_dispatch_rows_of_many_pairs(dtype, int8, tokens, topk, hidden, experts, total):
    g = gen(tokens)
    ids = routing(g, tokens, topk, total, 0.05)
    x = randn(g, tokens, hidden, dtype=dtype)
    _, order, slots, rows, scales = run_dispatch(ids, experts, 2, x, int8=int8, strided=True)
    want = torch.full((tokens * topk,), -1, dtype=torch.int32)
    kept = order >= 0
    want[order[kept].long()] = torch.arange(int(kept.sum()), dtype=torch.int32)
    assert torch.equal(slots.reshape(-1), want)
    codes, s = R.quant_i8(x) if int8 else (x, None)
    assert torch.equal(rows, R.gather(codes, order, topk))
    if int8:
        per_row = torch.ones(tokens * topk)
        per_row[kept] = s[order[kept].long() // topk]
        assert torch.equal(scales, per_row)


def special_rows(x):
    """Rows where quantizing can go wrong: all zero, one value, subnormal, near the largest, ties."""
    h = x.shape[1]
    x = x.clone()
    for i, v in enumerate((0.0, 1.0, 1e-40, 3e38)):
        if i < x.shape[0]:
            x[i] = v
    if x.shape[0] > 4:
        x[4] = torch.arange(h, dtype=FP32).remainder(255).sub(127).div(2).to(x.dtype)
        x[4, 0] = 127.0
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("tokens,topk,hidden", [(1, 1, 1), (6, 2, 9), (40, 8, 1030), (600, 8, 128), (7, 3, 20003)])
def test_dispatch_int8_rows(dtype, strided, tokens, topk, hidden):
    g = gen(hidden)
    ids = routing(g, tokens, topk, 16, 0.1)
    x = special_rows(randn(g, tokens, hidden, dtype=dtype, scale=3.0))
    _, order, _, rows, scales = run_dispatch(ids, 12, 0, x, int8=True, strided=strided)
    codes, s = R.quant_i8(x)
    assert torch.equal(rows, R.gather(codes, order, topk))
    want = torch.ones(tokens * topk)
    kept = order >= 0
    want[kept] = s[order[kept].long() // topk]
    assert torch.equal(scales, want)


# ---- combine -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,hidden,drop", [
    (1, 1, 1, 0.0), (1, 8, 8192, 0.0), (4, 2, 7, 0.5), (33, 8, 264, 0.2), (9, 12, 1001, 0.3), (6, 64, 72, 0.1),
    (5, 3, 20003, 0.2), (64, 4, 512, 1.0)])
def test_combine_and_backward(dtype, weighted, tokens, topk, hidden, drop):
    g = gen(hidden + topk)
    ids = routing(g, tokens, topk, 16 if topk < 16 else 64, drop)
    offsets, order, slots = R.plan(ids, 0, 12)
    kept, pairs = int(offsets[-1]), tokens * topk
    rows = randn(g, pairs, hidden, dtype=dtype)
    rows[kept:] = float("nan")   # what nobody owns is never read
    weights = torch.rand(tokens, topk, generator=g) if weighted else None
    if weighted:
        weights[slots < 0] = float("nan")   # nor is a dropped pair's weight used
    rg, out = put(Strided(pairs, hidden, dtype), rows), Strided(tokens, hidden, dtype)
    rx.rx_moe_combine(rg, gpu(slots), gpu(weights), out.t)
    want, bound = R.combine(rows, slots, weights)
    within(out.t, want, bound)
    out.check()

    d_out = randn(g, tokens, hidden, dtype=dtype)
    for with_dw in (True, False):
        d_rows = Strided(pairs, hidden, dtype)
        d_w = torch.full((tokens, topk), 77.0, device="cuda") if with_dw else None
        rx.rx_moe_combine_backward(put(Strided(tokens, hidden, dtype), d_out), rg if with_dw else None, gpu(slots),
                                   gpu(weights), gpu(offsets), d_rows.t, d_w)
        wr, br, ww, bw = R.combine_backward(d_out, rows, slots, weights, pairs)
        within(d_rows.t, wr, br)
        d_rows.check()
        if with_dw:
            within(d_w, ww, bw)


def test_combine_slots_past_the_rows_are_left_out():
    g = gen(1)
    rows = randn(g, 4, 16)
    slots = torch.tensor([[0, 4], [2 ** 31 - 1, 3], [-1, -5]], dtype=torch.int32)
    out = torch.empty(3, 16, device="cuda")
    rx.rx_moe_combine(rows.cuda(), slots.cuda(), None, out)
    assert torch.equal(out.cpu(), torch.stack([rows[0], rows[3], torch.zeros(16)]))


def test_combine_is_the_gradient_of_dispatch():
    g = gen(2)
    ids = routing(g, 50, 4, 10, 0.2)
    x = randn(g, 50, 96)
    offsets, order, slots, rows, _ = run_dispatch(ids, 10, 0, x)
    d_rows = randn(g, 200, 96)
    dx = torch.empty(50, 96, device="cuda")
    rx.rx_moe_combine(d_rows.cuda(), slots.cuda(), None, dx)
    xd = x.double().requires_grad_()
    kept = order >= 0
    (xd[order[kept].long() // 4] * d_rows.double()[kept]).sum().backward()
    _, bound = R.combine(d_rows, slots, None)
    within(dx, xd.grad, bound)


# ---- norm ----------------------------------------------------------------------

def norm_case(g, rows, hidden, nsrc, dtype, post, gate_rows, residual=True):
    groups = -(-rows // gate_rows) if gate_rows else 0
    return dict(srcs=[randn(g, rows, hidden, dtype=dtype) for _ in range(nsrc)],
                residual=randn(g, rows, hidden, dtype=dtype, scale=2.0) if residual else None,
                gate=randn(g, groups, hidden, dtype=dtype, scale=0.5) if groups else None,
                w_post=(1 + 0.1 * randn(g, hidden)).to(dtype) if post else None,
                w_pre=(1 + 0.1 * randn(g, hidden)).to(dtype)), groups


NORMS = [  # rows, hidden, sources, norm after the block, rows of a gate row (0: no gate)
    (1, 1, 1, True, 1), (1, 8192, 8, True, 1), (5, 7, 2, True, 2), (32, 264, 3, False, 0), (9, 1001, 16, True, 4),
    (300, 96, 5, True, 300), (1030, 72, 2, True, 700), (600, 40, 1, False, 3), (700, 130, 4, True, 1),
    (4, 5001, 6, True, 3), (3, 16384, 2, True, 2), (2, 32768, 1, True, 0), (3, 20003, 7, False, 1),
    # more rows than workgroups at each width that has a kernel of its own
    (530, 5203, 3, True, 130), (300, 9001, 2, True, 70), (300, 7000, 5, True, 0), (290, 12300, 1, False, 3), (259, 17000, 2, True, 100),
    (2100, 500, 9, True, 8), (2100, 1020, 2, True, 5), (3000, 64, 2, False, 1100)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,hidden,nsrc,post,gate_rows", NORMS)
def test_norm_and_backward(dtype, rows, hidden, nsrc, post, gate_rows):
    g = gen(rows + hidden)
    rs, eps = 0.75, 1e-5
    t, groups = norm_case(g, rows, hidden, nsrc, dtype, post, gate_rows)
    if rows > 3:   # a row of zeros, and one whose residual is zero
        for s in t["srcs"]:
            s[1] = 0
        t["residual"][1:3] = 0
    gr = gate_rows or 1
    f = R.norm(t["srcs"], t["residual"], t["gate"], gr, t["w_post"], t["w_pre"], rs, eps)
    srcs = [put(Strided(rows, hidden, dtype, extra=3), s) for s in t["srcs"]]
    res = put(Strided(rows, hidden, dtype, extra=9, shift=3), t["residual"])
    gate, wp, wz = gpu(t["gate"]), gpu(t["w_post"]), gpu(t["w_pre"])
    h, z = Strided(rows, hidden, dtype), Strided(rows, hidden, dtype)
    p, q = (torch.full((rows,), 77.0, device="cuda") for _ in range(2))
    rx.rx_residual_norm(srcs, res, gate, wp, wz, h.t, z.t, rstd_post=p if post else None, rstd_pre=q, gate_rows=gr,
                        residual_scale=rs, eps=eps)
    n = f["n"] * R.EPS32 * f["kappa"]
    within(h.t, f["h"], R.cast_bound(f["h"], n * f["hm"], dtype))
    within(z.t, f["z"], R.cast_bound(f["z"], n * f["zm"], dtype))
    within(q, f["q"][:, 0], (n * f["q"])[:, 0])
    if post:
        within(p, f["p"][:, 0], (n * f["p"])[:, 0])
    h.check(), z.check()

    d_h, d_z = randn(g, rows, hidden, dtype=dtype), randn(g, rows, hidden, dtype=dtype)
    d_src, d_res = Strided(rows, hidden, dtype), Strided(rows, hidden, dtype)
    new = lambda *s: torch.full(s, 77.0, device="cuda")
    d_gate = new(groups, hidden) if groups else None
    d_wp, d_wz = new(hidden) if post else None, new(hidden)
    ws = torch.full((rx.rx_residual_norm_backward_workspace(rows, hidden, gr),), 0xFF, dtype=torch.uint8, device="cuda")
    rx.rx_residual_norm_backward(srcs, res, gate, wp, wz, p if post else None, q, put(Strided(rows, hidden, dtype), d_h),
                                 put(Strided(rows, hidden, dtype), d_z), d_src.t, d_res.t, d_gate=d_gate, d_w_post=d_wp,
                                 d_w_pre=d_wz, gate_rows=gr, residual_scale=rs, workspace=ws)
    want = R.norm_backward(f, d_h, d_z, rs, post, groups)
    for name, got in (("d_src", d_src.t), ("d_residual", d_res.t), ("d_gate", d_gate), ("d_w_post", d_wp),
                      ("d_w_pre", d_wz)):
        if got is not None:
            value, err = want[name]
            within(got, value, R.cast_bound(value, err, got.dtype))
    d_src.check(), d_res.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", ["residual", "out_h", "out_z", "d_h", "d_z", "d_residual", "weights"])
def test_norm_optional_operands(dtype, drop):
    g = gen(8)
    rows, hidden, rs, eps = 70, 200, 1.5, 1e-6
    t, groups = norm_case(g, rows, hidden, 2, dtype, drop != "residual", 16, residual=drop != "residual")
    f = R.norm(t["srcs"], t["residual"], t["gate"], 16, t["w_post"], t["w_pre"], rs, eps)
    srcs = [gpu(s) for s in t["srcs"]]
    res, gate, wp, wz = (gpu(t[k]) for k in ("residual", "gate", "w_post", "w_pre"))
    new = lambda *s, dtype=FP32: torch.full(s, 77.0, dtype=dtype, device="cuda")
    h = new(rows, hidden, dtype=dtype) if drop != "out_h" else None
    z = new(rows, hidden, dtype=dtype) if drop != "out_z" else None
    p, q = new(rows), new(rows)
    rx.rx_residual_norm(srcs, res, gate, wp, wz if z is not None else None, h, z, rstd_post=p, rstd_pre=q, gate_rows=16,
                        residual_scale=rs, eps=eps)
    n = f["n"] * R.EPS32 * f["kappa"]
    if h is not None:
        within(h, f["h"], R.cast_bound(f["h"], n * f["hm"], dtype))
    if z is not None:
        within(z, f["z"], R.cast_bound(f["z"], n * f["zm"], dtype))
    if drop == "out_z":
        rx.rx_residual_norm(srcs, res, gate, wp, wz, None, new(rows, hidden, dtype=dtype), rstd_post=p, rstd_pre=q,
                            gate_rows=16, residual_scale=rs, eps=eps)
    d_h = randn(g, rows, hidden, dtype=dtype) if drop != "d_h" else None
    d_z = randn(g, rows, hidden, dtype=dtype) if drop != "d_z" else None
    d_src = new(rows, hidden, dtype=dtype)
    d_res = new(rows, hidden, dtype=dtype) if drop not in ("residual", "d_residual") else None
    keep = drop != "weights"
    d_gate = new(groups, hidden) if keep else None
    d_wp, d_wz = new(hidden) if keep and wp is not None else None, new(hidden) if keep else None
    ws = torch.empty(rx.rx_residual_norm_backward_workspace(rows, hidden, 16), dtype=torch.uint8, device="cuda")
    rx.rx_residual_norm_backward(srcs, res, gate, wp, wz, p if wp is not None else None, q if d_z is not None else None,
                                 gpu(d_h), gpu(d_z), d_src, d_res, d_gate=d_gate, d_w_post=d_wp, d_w_pre=d_wz,
                                 gate_rows=16, residual_scale=rs, workspace=ws)
    want = R.norm_backward(f, d_h, d_z, rs, wp is not None, groups)
    for name, got in (("d_src", d_src), ("d_residual", d_res), ("d_gate", d_gate), ("d_w_post", d_wp), ("d_w_pre", d_wz)):
        if got is not None:
            value, err = want[name]
            within(got, value, R.cast_bound(value, err, got.dtype))


def test_norm_in_place_and_no_rows():
    g = gen(9)
    t, _ = norm_case(g, 40, 520, 2, BF16, True, 0)
    srcs, res, wp, wz = [gpu(s) for s in t["srcs"]], gpu(t["residual"]), gpu(t["w_post"]), gpu(t["w_pre"])
    h, z, z2 = torch.empty_like(res), torch.empty_like(res), torch.empty_like(res)
    rx.rx_residual_norm(srcs, res, None, wp, wz, h, z)
    rx.rx_residual_norm(srcs, res, None, wp, wz, res, z2)
    assert torch.equal(res, h) and torch.equal(z, z2)
    none = torch.empty(0, 520, dtype=BF16, device="cuda")
    stat, d_w = torch.empty(0, device="cuda"), torch.full((520,), 7.0, device="cuda")
    rx.rx_residual_norm_backward([none], none, None, wp, wz, stat, stat, none, none, none.clone(), none.clone(), d_w_post=d_w)
    assert bool((d_w == 0).all())


# ---- INT8 ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 1), (6, 9), (40, 1030), (300, 128), (7, 20003), (64, 8192), (3, 0)])
def test_quant_i8(dtype, rows, k):
    x = special_rows(randn(gen(k), rows, k, dtype=dtype, scale=3.0)) if k else torch.zeros(rows, k, dtype=dtype)
    codes, scales = Strided(rows, k, torch.int8, extra=7), torch.empty(rows, device="cuda")
    rx.rx_quant_i8(put(Strided(rows, k, dtype), x), codes.t, scales)
    want, s = R.quant_i8(x)
    assert torch.equal(codes.t.cpu(), want) and torch.equal(scales.cpu(), s)
    codes.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [5, 520, 40000])
def test_quant_i8_rows_that_are_not_finite(dtype, k):
    x = torch.randn(4, k, generator=gen(k))
    x[0, 1], x[1, k - 1] = float("nan"), float("inf")
    x[2, 0], x[2, 2] = float("-inf"), float("nan")
    x = x.to(dtype)
    codes, scales = torch.full((4, k), 77, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    rx.rx_quant_i8(x.cuda(), codes, scales)
    want, s = R.quant_i8(x[3:])
    assert bool((codes[:3] == 0).all()) and torch.equal(codes[3:].cpu(), want) and torch.equal(scales[3:].cpu(), s)
    assert bool(scales[[0, 2]].isnan().all()) and float(scales[1]) == float("inf")
    _, order, _, rows, sc = run_dispatch(torch.tensor([[2], [0], [1], [3]], dtype=torch.int32), 4, 0, x, int8=True)
    at = order.argsort()   # the row of each token
    assert torch.equal(rows[at], codes.cpu()) and torch.equal(sc[at][[1, 3]], scales[[1, 3]].cpu())
    assert bool(sc[at][[0, 2]].isnan().all())


def padded(t, junk):
    """INT8 rows padded to 16 bytes with values that must not count."""
    k = t.shape[-1]
    full = torch.full((*t.shape[:-1], -(-k // 16) * 16 + 16), junk, dtype=torch.int8, device="cuda")
    full[..., :k] = t.cuda()
    return full[..., :k]


def i8(g, *shape):
    return torch.randint(-127, 128, shape, generator=g).to(torch.int8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 8192, 256), (2, 17, 100), (16, 16, 16), (17, 300, 127), (32, 512, 2048), (33, 129, 1025), (64, 64, 64),
    (65, 700, 640), (128, 128, 128), (129, 257, 384), (200, 1000, 8190), (300, 256, 1000), (513, 513, 272), (5, 40, 0),
    (260, 520, 65)])
def test_gemm_dense(dtype, m, n, k):
    g = gen(m + n + k)
    a, b = i8(g, m, k), i8(g, n, k)
    if k:
        a[0], b[0] = -127, -128   # the largest sums
    sa, sb = torch.rand(m, generator=g) + 0.5, torch.rand(n, generator=g) * 1e-3
    out = Strided(m, n, dtype)
    rx.rx_gemm_i8(padded(a, 99), gpu(sa), padded(b, -77), gpu(sb), out.t)
    want, bound = R.gemm_i8(a, sa, b, sb, dtype)
    within(out.t, want, bound)
    out.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,pad,n,k", [
    ([3], 0, 33, 48), ([0, 0, 0], 5, 20, 32), ([1, 0, 2, 0], 0, 300, 260), ([130, 0, 1, 257], 40, 200, 130),
    ([5] * 70, 0, 64, 64), ([0] * 65 + [9], 130, 70, 96), ([16, 17, 31, 32, 33], 3, 520, 1040), ([600, 100, 300], 0, 384, 512)])
def test_gemm_grouped(dtype, counts, pad, n, k):
    g = gen(sum(counts) + n)
    rows, experts = sum(counts) + pad, len(counts)
    a, b = i8(g, rows, k), i8(g, experts, n, k)
    sa, sb = torch.rand(rows, generator=g) + 0.5, torch.rand(experts, n, generator=g) * 1e-3
    sa[sum(counts):] = float("nan")   # rows past the last expert's are not used
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    out = Strided(rows, n, dtype)
    rx.rx_gemm_i8(padded(a, 99), gpu(sa), padded(b, -77), gpu(sb), out.t, offsets=gpu(offsets))
    want, bound = torch.zeros(rows, n, dtype=torch.float64), torch.zeros(rows, n, dtype=torch.float64)
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want[lo:hi], bound[lo:hi] = R.gemm_i8(a[lo:hi], sa[lo:hi], b[e], sb[e], dtype)
    within(out.t, want, bound)
    out.check()


TILES = [  # rows and columns that take each kind of tile, with partial ones
    (4090, 4090), (2041, 4090), (500, 8150), (250, 4100), (30, 4100)]


@pytest.mark.parametrize("m,n", TILES)
@pytest.mark.parametrize("k", [1, 16, 63, 65, 128, 129, 255, 300, 512, 1001])
def test_gemm_tiles(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + k)
    rnd = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
    a, b = padded(rnd(m, k), 99), padded(rnd(n, k), -77)
    a[-1], b[-1] = -127, -128
    sa, sb = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    out = Strided(m, n, FP32)
    rx.rx_gemm_i8(a, sa, b, sb, out.t)
    # sums below 2^24 are exact in float32
    assert torch.equal(out.t.double(), a.double() @ b.double().t())
    out.check()


@pytest.mark.parametrize("counts,pad,n,k", [
    ([700, 30, 0, 1500, 256, 1, 900], 9, 8001, 200), ([65, 1, 129, 250, 60, 0, 77, 128, 31, 200, 64, 65], 200, 4001, 333),
    ([128] * 9 + [1, 2, 3], 0, 1000, 260), ([9] * 30, 50, 700, 1025)])
def test_gemm_grouped_tiles(counts, pad, n, k):
    rows, experts = sum(counts) + pad, len(counts)
    g = torch.Generator(device="cuda").manual_seed(rows)
    rnd = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
    a, b = padded(rnd(rows, k), 99), padded(rnd(experts, n, k), -77)
    sa, sb = torch.ones(rows, device="cuda"), torch.ones(experts, n, device="cuda")
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    out = Strided(rows, n, FP32)
    rx.rx_gemm_i8(a, sa, b, sb, out.t, offsets=gpu(offsets))
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want[lo:hi] = a[lo:hi].double() @ b[e].double().t()
    assert torch.equal(out.t.double(), want)
    out.check()


def test_gemm_offsets_outside_the_rows_are_clamped():
    g = gen(5)
    a, b = i8(g, 20, 32), i8(g, 2, 24, 32)
    sa, sb = torch.ones(20), torch.ones(2, 24)
    out = Strided(20, 24, FP32)
    rx.rx_gemm_i8(a.cuda(), gpu(sa), b.cuda(), gpu(sb), out.t, offsets=torch.tensor([-4, 12, 900], dtype=torch.int32).cuda())
    want = torch.cat([a[:12].double() @ b[0].double().t(), a[12:].double() @ b[1].double().t()])
    assert torch.equal(out.t.cpu().double(), want)
    out.check()


def test_binding_refusals():
    z = lambda *s, dtype=FP32: torch.zeros(*s, dtype=dtype, device="cuda")
    x, codes, scales = z(4, 32), z(4, 32, dtype=torch.int8), z(4)
    refused = [
        (ValueError, "shape", lambda: rx.rx_quant_i8(x, z(4, 31, dtype=torch.int8), scales)),
        (TypeError, "Char", lambda: rx.rx_quant_i8(x, x, scales)),
        (ValueError, "rows must be contiguous", lambda: rx.rx_quant_i8(z(32, 4).t(), codes, scales)),
        (ValueError, "overlap", lambda: rx.rx_quant_i8(torch.as_strided(z(64), (4, 32), (8, 1)), codes, scales)),
        (ValueError, "scales must be contiguous", lambda: rx.rx_quant_i8(x, codes, z(8)[::2])),
        (ValueError, "GPU tensor", lambda: rx.rx_quant_i8(x, codes, scales.cpu())),
        (ValueError, "come together", lambda: rx.rx_moe_dispatch(z(4, 1, dtype=torch.int32), 2, z(3, dtype=torch.int32), z(4, dtype=torch.int32),
                                                                 z(4, 1, dtype=torch.int32), x=x)),
        (ValueError, "scales come with", lambda: rx.rx_moe_dispatch(z(4, 1, dtype=torch.int32), 2, z(3, dtype=torch.int32), z(4, dtype=torch.int32),
                                                                    z(4, 1, dtype=torch.int32), x=x, rows=codes)),
        (ValueError, "d_weights needs rows", lambda: rx.rx_moe_combine_backward(x, None, z(4, 1, dtype=torch.int32), None, z(3, dtype=torch.int32), x, z(4, 1))),
        (ValueError, "another row stride", lambda: rx.rx_residual_norm([x, z(4, 40)[:, :32]], None, None, None, None, x, None)),
        (ValueError, "gate_rows", lambda: rx.rx_residual_norm([x], None, z(1, 32), None, None, z(4, 32), None, gate_rows=0)),
        (ValueError, "padded", lambda: rx.rx_gemm_i8(torch.as_strided(z(3 * 48 + 40, dtype=torch.int8), (4, 40), (48, 1)), scales, z(8, 48, dtype=torch.int8)[:, :40],
                                                     z(8), z(4, 8))),
        (rx.RxError, "RX_ERR_ARG", lambda: rx.rx_residual_norm([x], None, None, None, None, z(4, 32), None, eps=0.0)),
    ]
    for error, match, call in refused:
        with pytest.raises(error, match=match):
            call()


# ---- far offsets, streams, graphs ------------------------------------------------

def test_row_offsets_past_32_bits():
    ld = (1 << 31) + 64
    g = gen(6)
    big = torch.empty(3 * ld, dtype=BF16, device="cuda")
    far = torch.as_strided(big, (3, 64), (ld, 1), 0)
    x = randn(g, 3, 64, dtype=BF16)
    far.copy_(x)
    rows = torch.empty(3, 64, dtype=BF16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    rx.rx_moe_dispatch(torch.tensor([[1], [0], [2]], **i32), 3, torch.empty(4, **i32), torch.empty(3, **i32),
                       torch.empty(3, 1, **i32), x=far, rows=rows)
    assert torch.equal(rows.cpu(), x[[1, 0, 2]])
    out = torch.empty(1, 64, dtype=BF16, device="cuda")
    rx.rx_moe_combine(far, torch.tensor([[2]], **i32), None, out)
    assert torch.equal(out.cpu(), x[2:])
    h = torch.empty(3, 64, dtype=BF16, device="cuda")
    rx.rx_residual_norm([far], None, None, None, None, h, None)
    assert torch.equal(h.cpu(), x)
    w = torch.as_strided(big.view(torch.int8), (2, 16, 64), (2 * ld, 64, 1), 0)
    wv = i8(g, 2, 16, 64)
    w.copy_(wv)
    a = i8(g, 4, 64)
    o = torch.empty(4, 16, device="cuda")
    rx.rx_gemm_i8(a.cuda(), torch.ones(4, device="cuda"), w, torch.ones(2, 16, device="cuda"), o,
                  offsets=torch.tensor([0, 1, 4], **i32))
    want = torch.cat([a[:1].double() @ wv[0].double().t(), a[1:].double() @ wv[1].double().t()])
    assert torch.equal(o.cpu().double(), want)


class Block:
    """Buffers of one pass through all operators, forward and backward."""

    def __init__(self, seed, tokens=48, topk=3, experts=6, hidden=136):
        g = gen(seed)
        self.ids = routing(g, tokens, topk, 9, 0.1).cuda()
        self.x, self.d_out, self.res, self.dz = (randn(g, tokens, hidden, dtype=BF16).cuda() for _ in range(4))
        self.weights = torch.rand(tokens, topk, generator=g).cuda()
        self.w = padded(i8(g, experts, hidden, hidden), 3)
        self.w_scales = (torch.rand(experts, hidden, generator=g) * 1e-3).cuda()
        self.norm_w = (1 + 0.1 * randn(g, hidden)).to(BF16).cuda()
        self.gate = randn(g, 1, hidden, dtype=BF16).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        pairs = tokens * topk
        self.offsets, self.order, self.slots = torch.zeros(experts + 1, **i32), torch.zeros(pairs, **i32), torch.zeros(tokens, topk, **i32)
        self.codes = padded(torch.zeros(pairs, hidden, dtype=torch.int8), 5)
        z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
        self.scales, self.y, self.out, self.h, self.z = z(pairs, dtype=FP32), z(pairs, hidden), z(tokens, hidden), z(tokens, hidden), z(tokens, hidden)
        self.p, self.q = z(tokens, dtype=FP32), z(tokens, dtype=FP32)
        self.d_src, self.d_res, self.d_rows = z(tokens, hidden), z(tokens, hidden), z(pairs, hidden)
        self.d_w, self.d_gate, self.d_wp, self.d_wz = z(tokens, topk, dtype=FP32), z(1, hidden, dtype=FP32), z(hidden, dtype=FP32), z(hidden, dtype=FP32)
        self.ws = z(rx.rx_residual_norm_backward_workspace(tokens, hidden), dtype=torch.uint8)
        self.experts = experts

    def run(self):
        rx.rx_moe_dispatch(self.ids, self.experts, self.offsets, self.order, self.slots, x=self.x, rows=self.codes, scales=self.scales, first_expert=1)
        rx.rx_gemm_i8(self.codes, self.scales, self.w, self.w_scales, self.y, offsets=self.offsets)
        rx.rx_moe_combine(self.y, self.slots, self.weights, self.out)
        rx.rx_residual_norm([self.out], self.res, self.gate, self.norm_w, self.norm_w, self.h, self.z, rstd_post=self.p, rstd_pre=self.q)
        rx.rx_residual_norm_backward([self.out], self.res, self.gate, self.norm_w, self.norm_w, self.p, self.q, self.d_out, self.dz, self.d_src,
                                     self.d_res, d_gate=self.d_gate, d_w_post=self.d_wp, d_w_pre=self.d_wz, workspace=self.ws)
        rx.rx_moe_combine_backward(self.d_src, self.y, self.slots, self.weights, self.offsets, self.d_rows, self.d_w)

    def results(self):
        return [t.clone() for t in (self.offsets, self.order, self.slots, self.codes, self.scales, self.y, self.out, self.h, self.z, self.d_src,
                                    self.d_res, self.d_gate, self.d_wp, self.d_wz, self.d_rows, self.d_w)]


def test_block_on_another_stream_and_in_a_graph():
    b, other = Block(1), Block(2)
    b.run()
    torch.cuda.synchronize()
    want = b.results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
        got = b.results()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for _ in range(4):
        for t in (b.y, b.out, b.h, b.z, b.d_src, b.d_rows, b.d_w, b.d_gate, b.ws, b.offsets):
            t.zero_()
        other.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(b.results(), want))
