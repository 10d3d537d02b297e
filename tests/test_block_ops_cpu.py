"""The operators around a block's allreduce without a GPU: the C entry points'
refusals (nothing is launched: every call fails validation or has nothing to
do), the binding's refusals, and the float64 reference's gradients against
differences of its forward pass."""
import ctypes

import pytest
import torch

import allreduce_reduction_rx_amd as rx
import block_ref as R

OK, NULL, ARG, DTYPE, ALIGN = 0, 1, 2, 3, 4
F = 0x7F0000000000   # aligned, never dereferenced
FP32, BF16, I8 = rx.RX_FP32, rx.RX_BF16, rx.RX_INT8


def ptrs(*vals):
    return (ctypes.c_void_p * max(1, len(vals)))(*vals)


def dispatch(ids=F, tokens=4, topk=2, first=0, experts=8, x=F, ldx=64, hidden=64, xdt=BF16, offsets=F, order=F,
             slots=F, rows=F, ldr=64, rdt=BF16, scales=None, ws=None, wsb=0):
    return rx.lib().rx_moe_dispatch(ids, tokens, topk, first, experts, x, ldx, hidden, xdt, offsets, order, slots,
                                    rows, ldr, rdt, scales, ws, wsb, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(offsets=None)), (NULL, dict(ids=None)), (NULL, dict(order=None)), (NULL, dict(slots=None)),
    (NULL, dict(x=None)), (NULL, dict(rows=None)), (NULL, dict(rdt=I8)),
    (ARG, dict(topk=0)), (ARG, dict(topk=65)), (ARG, dict(experts=0)), (ARG, dict(experts=1025)),
    (ARG, dict(first=-1)), (ARG, dict(first=2 ** 31 - 4)), (ARG, dict(tokens=1 << 22)), (ARG, dict(ldx=63)),
    (ARG, dict(ldr=63)), (ARG, dict(scales=F)), (ARG, dict(hidden=(1 << 30) + 1, ldx=1 << 31, ldr=1 << 31)),
    (DTYPE, dict(xdt=rx.RX_FP8_E4M3)), (DTYPE, dict(rdt=FP32)), (DTYPE, dict(xdt=9)),
    (ALIGN, dict(x=F + 1)), (ALIGN, dict(rows=F + 1)), (ALIGN, dict(offsets=F + 2)), (ALIGN, dict(slots=F + 1)),
    (ALIGN, dict(rdt=I8, scales=F + 2)),
    (NULL, dict(tokens=4096)), (ARG, dict(tokens=4096, ws=F, wsb=4)), (ALIGN, dict(tokens=4096, ws=F + 1, wsb=1 << 20)),
])
def test_dispatch_refusals(want, kw):
    assert dispatch(**kw) == want


def test_dispatch_workspace():
    assert rx.rx_moe_dispatch_workspace(16, 8, 64) == 0
    assert rx.rx_moe_dispatch_workspace(16384, 8, 64) >= 64 * 4 * 129
    assert rx.rx_moe_dispatch_workspace(16, 0, 64) == 0


def combine(rows=F, ldr=64, nrows=8, slots=F, weights=F, tokens=4, topk=2, hidden=64, dt=BF16, out=F, ldo=64):
    return rx.lib().rx_moe_combine(rows, ldr, nrows, slots, weights, tokens, topk, hidden, dt, out, ldo, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(rows=None)), (NULL, dict(slots=None)), (NULL, dict(out=None)),
    (ARG, dict(topk=0)), (ARG, dict(topk=65)), (ARG, dict(ldr=8)), (ARG, dict(ldo=8)), (ARG, dict(nrows=1 << 31)),
    (ARG, dict(tokens=1 << 22)), (ARG, dict(tokens=1 << 21, hidden=1 << 20, ldr=1 << 20, ldo=1 << 20)),
    (DTYPE, dict(dt=I8)), (ALIGN, dict(rows=F + 1)), (ALIGN, dict(dt=FP32, out=F + 2)), (ALIGN, dict(weights=F + 2)),
    (OK, dict(tokens=0)), (OK, dict(hidden=0)),
])
def test_combine_refusals(want, kw):
    assert combine(**kw) == want


def combine_bwd(g=F, ldg=64, rows=F, ldr=64, nrows=8, slots=F, weights=F, kept=F, tokens=4, topk=2, hidden=64,
                dt=BF16, dr=F, lddr=64, dw=F):
    return rx.lib().rx_moe_combine_backward(g, ldg, rows, ldr, nrows, slots, weights, kept, tokens, topk, hidden, dt,
                                            dr, lddr, dw, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(g=None)), (NULL, dict(rows=None)), (NULL, dict(slots=None)), (NULL, dict(kept=None)),
    (NULL, dict(dr=None)), (ARG, dict(topk=0)), (ARG, dict(ldg=8)), (ARG, dict(ldr=8)), (ARG, dict(lddr=8)),
    (DTYPE, dict(dt=rx.RX_FP8_E5M2)), (ALIGN, dict(g=F + 1)), (ALIGN, dict(kept=F + 2)), (ALIGN, dict(dw=F + 1)),
    (OK, dict(tokens=0)),
])
def test_combine_backward_refusals(want, kw):
    assert combine_bwd(**kw) == want


def norm(srcs="two", nsrc=2, lds=64, res=F, ldr=64, gate=F, gr=4, wpost=F, wpre=F, rs=1.0, eps=1e-6, rows=4,
         hidden=64, dt=BF16, h=F, ldh=64, z=F, ldz=64, rp=F, rq=F):
    p = {"two": ptrs(F, F + 4096), "null": ptrs(F, 0), "odd": ptrs(F, F + 1), None: None}[srcs]
    return rx.lib().rx_residual_norm(p, nsrc, lds, res, ldr, gate, gr, wpost, wpre, rs, eps, rows, hidden, dt, h, ldh,
                                     z, ldz, rp, rq, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(srcs=None)), (NULL, dict(srcs="null")), (NULL, dict(h=None, z=None)), (NULL, dict(wpre=None)),
    (ARG, dict(nsrc=0)), (ARG, dict(nsrc=17)), (ARG, dict(lds=63)), (ARG, dict(ldr=63)), (ARG, dict(ldh=63)),
    (ARG, dict(ldz=63)), (ARG, dict(gr=0)), (ARG, dict(eps=0.0)), (ARG, dict(eps=float("nan"))),
    (ARG, dict(eps=float("inf"))), (ARG, dict(rs=float("inf"))), (ARG, dict(rows=1 << 22)),
    (ARG, dict(hidden=32769, lds=40000, ldr=40000, ldh=40000, ldz=40000)),
    (DTYPE, dict(dt=I8)), (ALIGN, dict(srcs="odd")), (ALIGN, dict(gate=F + 1)), (ALIGN, dict(rq=F + 2)),
    (OK, dict(rows=0)), (OK, dict(hidden=0)),
])
def test_norm_refusals(want, kw):
    assert norm(**kw) == want


def norm_bwd(srcs="two", nsrc=2, lds=64, res=F, ldr=64, gate=F, gr=4, wpost=F, wpre=F, rp=F, rq=F, rs=1.0, rows=4,
             hidden=64, dt=BF16, dh=F, lddh=64, dz=F, lddz=64, ds=F, ldds=64, dr=F, lddr=64, dg=F, dwp=F, dwq=F, ws=F,
             wsb=1 << 30):
    p = {"two": ptrs(F, F + 4096), "null": ptrs(F, 0), None: None}[srcs]
    return rx.lib().rx_residual_norm_backward(p, nsrc, lds, res, ldr, gate, gr, wpost, wpre, rp, rq, rs, rows, hidden,
                                              dt, dh, lddh, dz, lddz, ds, ldds, dr, lddr, dg, dwp, dwq, ws, wsb, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(srcs=None)), (NULL, dict(srcs="null")), (NULL, dict(ds=None)), (NULL, dict(rq=None)),
    (NULL, dict(rp=None)), (NULL, dict(wpre=None)), (NULL, dict(ws=None)), (ARG, dict(wsb=16)),
    (ARG, dict(res=None)), (ARG, dict(gate=None)), (ARG, dict(wpost=None)), (ARG, dict(dz=None, wpre=None)),
    (ARG, dict(lddh=8)), (ARG, dict(lddz=8)), (ARG, dict(ldds=8)), (ARG, dict(lddr=8)), (ARG, dict(gr=0)),
    (DTYPE, dict(dt=I8)), (ALIGN, dict(ds=F + 1)), (ALIGN, dict(ws=F + 4)), (ALIGN, dict(dg=F + 2)),
])
def test_norm_backward_refusals(want, kw):
    assert norm_bwd(**kw) == want


def quant(x=F, ldx=64, rows=4, k=64, dt=BF16, codes=F, ldc=64, scales=F):
    return rx.lib().rx_quant_i8(x, ldx, rows, k, dt, codes, ldc, scales, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(codes=None)), (NULL, dict(scales=None)), (ARG, dict(ldx=8)), (ARG, dict(ldc=8)),
    (ARG, dict(rows=1 << 22)), (DTYPE, dict(dt=I8)), (ALIGN, dict(x=F + 1)), (ALIGN, dict(scales=F + 2)),
    (OK, dict(rows=0)),
])
def test_quant_i8_refusals(want, kw):
    assert quant(**kw) == want


def gemm(a=F, lda=64, sa=F, b=F, ldb=64, stride=0, sb=F, offsets=None, experts=1, rows=4, n=8, k=64, out=F, ldo=8,
         dt=BF16):
    return rx.lib().rx_gemm_i8(a, lda, sa, b, ldb, stride, sb, offsets, experts, rows, n, k, out, ldo, dt, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(a=None)), (NULL, dict(b=None)), (NULL, dict(sa=None)), (NULL, dict(sb=None)), (NULL, dict(out=None)),
    (ARG, dict(experts=0)), (ARG, dict(experts=2)), (ARG, dict(offsets=F, experts=1025)), (ARG, dict(lda=48)),
    (ARG, dict(ldb=48)), (ARG, dict(k=50, lda=50)), (ARG, dict(ldo=7)), (ARG, dict(k=131072, lda=131072, ldb=131072)),
    (ARG, dict(rows=1 << 22)), (DTYPE, dict(dt=I8)), (ALIGN, dict(a=F + 8)), (ALIGN, dict(lda=72)),
    (ALIGN, dict(offsets=F, stride=520)), (ALIGN, dict(out=F + 1)), (OK, dict(rows=0)), (OK, dict(n=0)),
])
def test_gemm_refusals(want, kw):
    assert gemm(**kw) == want


@pytest.mark.parametrize("kw", [dict(lda=1 << 23), dict(ldb=1 << 23), dict(rows=1 << 21, n=1 << 21, ldo=1 << 21)])
def test_gemm_refuses_what_its_tiles_cannot_address(kw):
    assert gemm(**kw) == ARG


def test_binding_refuses_cpu_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_quant_i8(x, torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_residual_norm([x], x, None, None, None, x, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_moe_combine(x, torch.zeros(2, 2, dtype=torch.int32), None, torch.zeros(2, 8))


def test_binding_refuses_what_is_no_matrix(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError, match="x must be a tensor"):
        rx.rx_quant_i8(5, x, x)
    with pytest.raises(ValueError, match="two dimensions"):
        rx.rx_quant_i8(torch.zeros(2, 3, 4), x, x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        rx.rx_quant_i8(i, x, x)
    with pytest.raises(ValueError, match="1 to 16 sources"):
        rx.rx_residual_norm([], x, None, None, None, x, None)
    with pytest.raises(ValueError, match="1 to 16 sources"):
        rx.rx_residual_norm([x] * 17, x, None, None, None, x, None)
    with pytest.raises(TypeError, match="sequence"):
        rx.rx_residual_norm(3, x, None, None, None, x, None)
    with pytest.raises(ValueError, match="b must have three dimensions"):
        rx.rx_gemm_i8(x, x, x, x, x, offsets=i)
    with pytest.raises(ValueError, match="32 bits"):
        rx.rx_moe_dispatch(i, 1 << 40, i, i, i)
    with pytest.raises(TypeError):
        rx.rx_moe_dispatch(i, "eight", i, i, i)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate_rows", [0, 2, 5])
def test_reference_norm_gradient_against_differences(post, gate_rows):
    gen = torch.Generator().manual_seed(3)
    rows, hidden, rs, eps = 5, 7, 0.6, 1e-3
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    groups = -(-rows // gate_rows) if gate_rows else 0
    t = dict(src=rnd(rows, hidden), residual=rnd(rows, hidden), gate=rnd(groups, hidden) if groups else None,
             w_post=rnd(hidden) if post else None, w_pre=rnd(hidden))
    other, dh, dz = rnd(rows, hidden), rnd(rows, hidden), rnd(rows, hidden)

    def forward(t):
        return R.norm([t["src"], other], t["residual"], t["gate"], max(1, gate_rows), t["w_post"], t["w_pre"], rs, eps)

    grads = R.norm_backward(forward(t), dh, dz, rs, post, groups)
    step = 1e-5
    for name in t:
        if t[name] is None:
            continue
        dirn = rnd(*t[name].shape)
        vals = []
        for sign in (1, -1):
            f = forward(dict(t, **{name: t[name] + sign * step * dirn}))
            vals.append(((f["h"] * dh).sum() + (f["z"] * dz).sum()).item())
        want = (vals[0] - vals[1]) / (2 * step)
        got = (grads["d_" + name][0] * dirn).sum().item()
        # truncation step^2 times third derivatives of order 100, rounding 1e-16 * 100 / step
        assert abs(got - want) < 1e-7 * max(1.0, abs(want)), name


def test_reference_combine_gradient_against_differences():
    gen = torch.Generator().manual_seed(4)
    ids = torch.tensor([[0, 2], [1, -1], [-1, -1], [2, 0]], dtype=torch.int32)
    _, _, slots = R.plan(ids, 0, 3)
    rows, w, g = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((8, 5), (4, 2), (4, 5)))
    R.HALF[torch.float64] = 0.0
    d_rows, _, d_w, _ = R.combine_backward(g, rows, slots, w, 8)
    step = 1e-3   # the form is linear in each argument: no truncation
    for arg, grad in (("rows", d_rows), ("w", d_w)):
        dirn = torch.randn(*grad.shape, generator=gen, dtype=torch.float64)
        f = lambda e: (R.combine(rows + e * dirn if arg == "rows" else rows, slots,
                                 w + e * dirn if arg == "w" else w)[0] * g).sum().item()
        assert abs((f(step) - f(-step)) / (2 * step) - (grad * dirn).sum().item()) < 1e-10
