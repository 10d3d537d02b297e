"""The operators around a block's allreduce at the edges of what their calls
accept, against their float64 forms (block_ref.py)."""
import pytest
import torch

import allreduce_reduction_rx_amd as rx
import block_ref as R
from test_block_ops_gpu import BF16, DTYPES, FP32, Strided, gen, gpu, norm_case, put, randn, routing, run_dispatch, within

pytestmark = pytest.mark.gpu


# ---- norm: rows of any size ------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("hidden", [136, 16400, 20000])   # registers, 1024 threads or long rows, long rows
@pytest.mark.parametrize("scale,eps", [(1e16, 1e-5), (1e14, 1e-5), (1e-13, 1e-30), (1e-15, 1e-30), (1.0, 1e-30)])
def test_norm_gradient_of_rows_far_from_one(scale, eps, hidden, post, dtype):
    """Rows whose size, cubed, is no float32, and rows of zeros whose statistic is 1 / sqrt(eps). The bounds
    count relative roundings; every value on the way is a normal float32."""
    g = gen(hidden)
    rows, rs, eps = 9, 0.75, torch.tensor(eps).item()   # eps: the float32 that the call gets
    t, groups = norm_case(g, rows, hidden, 2, dtype, post, 4)
    t["srcs"] = [(s.double() * scale).to(dtype) for s in t["srcs"]]
    t["residual"] = (t["residual"].double() * scale).to(dtype)
    for s in (*t["srcs"], t["residual"]):
        s[5] = 0
    f = R.norm(t["srcs"], t["residual"], t["gate"], 4, t["w_post"], t["w_pre"], rs, eps)
    srcs, res, gate, wp, wz = [gpu(s) for s in t["srcs"]], *(gpu(t[k]) for k in ("residual", "gate", "w_post", "w_pre"))
    new = lambda *s, dtype=FP32: torch.full(s, 77.0, dtype=dtype, device="cuda")
    h, z, d_src, d_res = (new(rows, hidden, dtype=dtype) for _ in range(4))
    p, q = new(rows), new(rows)
    rx.rx_residual_norm(srcs, res, gate, wp, wz, h, z, rstd_post=p if post else None, rstd_pre=q, gate_rows=4,
                        residual_scale=rs, eps=eps)
    n = f["n"] * R.EPS32 * f["kappa"]
    within(h, f["h"], R.cast_bound(f["h"], n * f["hm"], dtype))
    within(z, f["z"], R.cast_bound(f["z"], n * f["zm"], dtype))
    within(q, f["q"][:, 0], (n * f["q"])[:, 0])

    d_z = randn(g, rows, hidden, dtype=dtype)
    d_gate, d_wp, d_wz = new(groups, hidden), new(hidden) if post else None, new(hidden)
    ws = torch.full((rx.rx_residual_norm_backward_workspace(rows, hidden, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    rx.rx_residual_norm_backward(srcs, res, gate, wp, wz, p if post else None, q, None, gpu(d_z), d_src, d_res,
                                 d_gate=d_gate, d_w_post=d_wp, d_w_pre=d_wz, gate_rows=4, residual_scale=rs, workspace=ws)
    want = R.norm_backward(f, None, d_z, rs, post, groups)
    for name, got in (("d_src", d_src), ("d_residual", d_res), ("d_gate", d_gate), ("d_w_post", d_wp), ("d_w_pre", d_wz)):
        if got is not None:
            value, err = want[name]
            within(got, value, R.cast_bound(value, err, got.dtype))


# ---- combine: no tokens ------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [1, 7, 264, 4100])
@pytest.mark.parametrize("nrows,kept", [(1, 0), (5, 0), (5, 3), (5, 5), (3000, 0), (3000, 2999), (4, 9), (0, 0)])
def test_combine_gradient_without_tokens(nrows, kept, hidden, dtype):
    """A rank whose tokens went elsewhere, with a row buffer of its own size: rows from kept on are 0."""
    i32 = dict(dtype=torch.int32, device="cuda")
    d_rows = Strided(nrows, hidden, dtype)
    offsets = torch.tensor([0, kept], **i32)
    empty = torch.empty(0, hidden, dtype=dtype, device="cuda")
    for rows, d_w in ((None, None), (torch.ones(nrows, hidden, dtype=dtype, device="cuda"), torch.empty(0, 2, device="cuda"))):
        d_rows.full.fill_(77.0)
        rx.rx_moe_combine_backward(empty, rows, torch.empty(0, 2, **i32), None, offsets, d_rows.t, d_w)
        assert bool((d_rows.t[kept:] == 0).all()) and bool((d_rows.t[:kept] == 77).all())
        d_rows.check()


# ---- dispatch: a workgroup of one wave ------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,topk", [(1, 1), (7, 2), (8, 8), (1, 64), (4, 16), (13, 5)])   # 64 pairs and one more
@pytest.mark.parametrize("hidden", [1, 250, 256, 257, 512, 513])                 # 64 vectors and one more
def test_dispatch_int8_of_few_pairs_and_short_rows(tokens, topk, hidden, dtype):
    """Rows whose largest value one wave finds alone, and those that several find together."""
    g = gen(tokens + hidden)
    ids = routing(g, tokens, topk, 64)
    x = randn(g, tokens, hidden, dtype=dtype) * (1 + torch.arange(tokens))[:, None].to(dtype)
    _, order, _, rows, scales = run_dispatch(ids, 50, 3, x, int8=True)
    codes, s = R.quant_i8(x)
    kept = order >= 0
    assert torch.equal(rows, R.gather(codes, order, topk))
    assert torch.equal(scales[kept], s[order[kept].long() // topk]) and bool((scales[~kept] == 1).all())


# ---- the binding: who holds the sources ---------------------------------------------------

def test_sources_of_a_generator_live_until_the_launch():
    """The stream is looked up after the checks and before the launch: the tensors that only a generator had
    must hold their memory then, and no longer after the call."""
    import ctypes

    g = gen(31)
    data = [randn(g, 4, 96) for _ in range(3)]
    h, want = torch.empty(4, 96, device="cuda"), torch.empty(4, 96, device="cuda")
    rx.rx_residual_norm([t.cuda() for t in data], None, None, None, None, want, None)
    L, m, held = rx.lib(), rx._bind(), []
    at = [ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
        "rx_moe_dispatch", "rx_moe_combine", "rx_moe_combine_backward", "rx_residual_norm", "rx_residual_norm_backward",
        "rx_quant_i8", "rx_gemm_i8")]
    before = torch.cuda.memory_allocated()

    def stream(device):
        held.append(torch.cuda.memory_allocated() - before)
        return torch._C._cuda_getCurrentRawStream(device)

    try:
        m.connect(stream, *at)
        rx.rx_residual_norm((t.cuda() for t in data), None, None, None, None, h, None)
    finally:
        m.connect(torch._C._cuda_getCurrentRawStream, *at)
    assert len(held) == 1 and held[0] >= 3 * 4 * 96 * 4
    assert torch.cuda.memory_allocated() == before and torch.equal(h, want)


# ---- the binding: one row, no columns ----------------------------------------------------

def test_one_row_has_no_stride():
    """A single token's row, cut out of buffers of different widths."""
    g = gen(21)
    wide = [torch.zeros(1, 64 + 8 * j, dtype=BF16, device="cuda")[:, :64] for j in range(3)]
    for t in wide:
        t.copy_(randn(g, 1, 64, dtype=BF16))
    far = torch.as_strided(wide[0], (1, 64), (1, 1))   # a row's own stride may be any number
    h, want = torch.empty(1, 64, dtype=BF16, device="cuda"), torch.empty(1, 64, dtype=BF16, device="cuda")
    rx.rx_residual_norm([far, *wide[1:]], None, None, None, None, h, None)
    rx.rx_residual_norm([t.contiguous() for t in wide], None, None, None, None, want, None)
    assert torch.equal(h, want)


@pytest.mark.parametrize("grouped", [False, True])
def test_gemm_of_one_row_and_one_channel(grouped):
    g = gen(22)
    a, b = (torch.randint(-127, 128, (112,), generator=g).to(torch.int8).cuda() for _ in range(2))
    va, vb = a[:100].unsqueeze(0), b[:100].unsqueeze(0)   # strides of 100, rows padded to 112
    one, out = torch.ones(1, device="cuda"), torch.empty(1, 1, device="cuda")
    if grouped:
        rx.rx_gemm_i8(va, one, vb.unsqueeze(0), one.view(1, 1), out, offsets=torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    else:
        rx.rx_gemm_i8(va, one, vb, one, out)
    assert out.item() == (a[:100].double() @ b[:100].double()).item()


@pytest.mark.parametrize("grouped", [False, True])
def test_gemm_without_columns_gives_zeros(grouped):
    i8 = dict(dtype=torch.int8, device="cuda")
    out = torch.full((5, 3), 77.0, device="cuda")
    if grouped:
        rx.rx_gemm_i8(torch.empty(5, 0, **i8), torch.ones(5, device="cuda"), torch.empty(2, 3, 0, **i8), torch.ones(2, 3, device="cuda"), out,
                      offsets=torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"))
    else:
        rx.rx_gemm_i8(torch.empty(5, 0, **i8), torch.ones(5, device="cuda"), torch.empty(3, 0, **i8), torch.ones(3, device="cuda"), out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate_len", [0, 1])
def test_norm_without_rows_keeps_the_gate(gate_len, dtype):
    """A gate for all rows is one row, also where there are none: its gradient is an empty sum."""
    none = lambda: torch.empty(0, 72, dtype=dtype, device="cuda")
    gate, w = torch.ones(gate_len, 72, dtype=dtype, device="cuda"), torch.ones(72, dtype=dtype, device="cuda")
    stat = torch.empty(0, device="cuda")
    rx.rx_residual_norm([none()], none(), gate, w, w, none(), none(), rstd_post=stat, rstd_pre=stat)
    d = [torch.full(s, 77.0, device="cuda") for s in ((gate_len, 72), (72,), (72,))]
    rx.rx_residual_norm_backward([none()], none(), gate, w, w, stat, stat, none(), none(), none(), none(), d_gate=d[0],
                                 d_w_post=d[1], d_w_pre=d[2])
    assert all(bool((t == 0).all()) for t in d)
    with pytest.raises(ValueError, match="shape"):
        rx.rx_residual_norm([none()], None, torch.ones(2, 72, dtype=dtype, device="cuda"), None, None, none(), None)


# ---- promises of aliasing ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("rows,hidden,nsrc", [(3, 7, 2), (40, 520, 3), (300, 1001, 2), (4, 5001, 9), (2, 20003, 2), (2, 32768, 5)])
def test_norm_in_place(rows, hidden, nsrc, post, dtype):
    """out_h in any source or the residual, d_residual in d_h: the same bits as in buffers of their own."""
    g = gen(rows + hidden)
    t, _ = norm_case(g, rows, hidden, nsrc, dtype, post, 1)
    mat = lambda v: put(Strided(rows, hidden, dtype, extra=3), v)
    gate, wp, wz = (gpu(t[k]) for k in ("gate", "w_post", "w_pre"))
    p, q = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def forward(into):
        ts = [mat(v) for v in (*t["srcs"], t["residual"])]
        h, z = Strided(rows, hidden, dtype).t if into is None else ts[into], Strided(rows, hidden, dtype).t
        rx.rx_residual_norm(ts[:-1], ts[-1], gate, wp, wz, h, z, rstd_post=p if post else None, rstd_pre=q, gate_rows=1)
        return h, z

    h, z = forward(None)
    for into in range(nsrc + 1):
        got_h, got_z = forward(into)
        assert torch.equal(got_h, h) and torch.equal(got_z, z), into

    d_h, d_z = randn(g, rows, hidden, dtype=dtype), randn(g, rows, hidden, dtype=dtype)
    ws = torch.empty(rx.rx_residual_norm_backward_workspace(rows, hidden, 1), dtype=torch.uint8, device="cuda")
    srcs, res = [mat(s) for s in t["srcs"]], mat(t["residual"])

    def backward(in_place):
        dh, ds = mat(d_h), mat(torch.zeros_like(d_h))
        dr = dh if in_place else mat(torch.zeros_like(d_h))
        grads = [torch.empty(s, device="cuda") for s in ((rows, hidden), (hidden,), (hidden,))]
        rx.rx_residual_norm_backward(srcs, res, gate, wp, wz, p if post else None, q, dh, mat(d_z), ds, dr, d_gate=grads[0],
                                     d_w_post=grads[1] if post else None, d_w_pre=grads[2], gate_rows=1, workspace=ws)
        return [ds, dr, grads[0], grads[2]] + grads[1:2] * post

    assert all(torch.equal(a, b) for a, b in zip(backward(True), backward(False)))


# ---- products: more experts than a wave has lanes -------------------------------------------

@pytest.mark.parametrize("experts,every,most", [(64, 1, 3), (65, 64, 40), (128, 127, 300), (1024, 1, 2), (1000, 333, 70)])
def test_gemm_of_many_experts(experts, every, most):
    """Experts with and without rows past the first 64, whose offsets are looked up in turns."""
    g = gen(experts)
    counts = [int(torch.randint(0, most + 1, (1,), generator=g)) if e % every == 0 or e == experts - 1 else 0 for e in range(experts)]
    rows, n, k = sum(counts) + 3, 24, 40
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    a, b = (torch.randint(-127, 128, s, generator=g).to(torch.int8) for s in ((rows, 48), (experts, n, 48)))
    out = Strided(rows, n, FP32)
    rx.rx_gemm_i8(gpu(a)[:, :k], torch.ones(rows, device="cuda"), gpu(b)[:, :, :k], torch.ones(experts, n, device="cuda"), out.t,
                  offsets=gpu(offsets))
    expert = torch.repeat_interleave(torch.arange(experts), torch.tensor(counts))
    want = torch.zeros(rows, n, dtype=torch.float64)
    want[:-3] = (b[expert][:, :, :k].double() * a[:-3, None, :k].double()).sum(2)
    assert torch.equal(out.t.cpu().double(), want)   # sums below 2^24: exact in float32
    out.check()
