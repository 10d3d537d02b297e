"""The router, the products with 4-bit weights and the layer norm without a GPU:
the C entry points' refusals (nothing is launched), the binding's refusals, the
float64 references' gradients against differences, and the reference generator
against the published numbers."""
import ctypes

import numpy as np
import pytest
import torch

import allreduce_reduction_rx_amd as rx
import block_ref as B
import layer_ref as R

OK, NULL, ARG, DTYPE, ALIGN = 0, 1, 2, 3, 4
F = 0x7F0000000000   # aligned, never dereferenced
FP32, BF16, I8 = rx.RX_FP32, rx.RX_BF16, rx.RX_INT8
NAN = float("nan")


def ptrs(*vals):
    return (ctypes.c_void_p * max(1, len(vals)))(*vals)


def route(logits=F, ld=64, mask=None, tokens=4, experts=64, topk=2, renorm=0, dt=BF16, ids=F, weights=F, lse=None,
          counts=None, losses=None, ws=None, wsb=0):
    return rx.lib().rx_moe_route(logits, ld, mask, tokens, experts, topk, renorm, dt, ids, weights, lse, counts, losses, ws, wsb, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(logits=None)), (NULL, dict(ids=None)), (NULL, dict(weights=None)), (NULL, dict(counts=F)), (NULL, dict(losses=F)),
    (ARG, dict(experts=0)), (ARG, dict(experts=1025, ld=2048)), (ARG, dict(topk=0)), (ARG, dict(topk=65)),
    (ARG, dict(experts=4, topk=5)), (ARG, dict(ld=63)), (ARG, dict(tokens=1 << 22)), (ARG, dict(ld=(1 << 36) + 1)),
    (DTYPE, dict(dt=I8)), (DTYPE, dict(dt=9)), (ALIGN, dict(logits=F + 1)), (ALIGN, dict(dt=FP32, logits=F + 2)),
    (ALIGN, dict(ids=F + 2)), (ALIGN, dict(weights=F + 1)), (ALIGN, dict(lse=F + 2)),
    (NULL, dict(counts=F, losses=F)), (ALIGN, dict(counts=F, losses=F, ws=F + 2, wsb=1 << 30)),
    (ARG, dict(counts=F, losses=F, ws=F, wsb=8)), (OK, dict(tokens=0, logits=None, ids=None, weights=None)),
])
def test_route_refusals(want, kw):
    assert route(**kw) == want


def route_backward(logits=F, ld=64, ids=F, lse=F, counts=F, dw=F, dl=F, tokens=4, experts=64, topk=2, renorm=0, dt=BF16, out=F, ldo=64):
    return rx.lib().rx_moe_route_backward(logits, ld, ids, lse, counts, dw, dl, tokens, experts, topk, renorm, dt, out, ldo, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(logits=None)), (NULL, dict(ids=None)), (NULL, dict(lse=None)), (NULL, dict(counts=None)), (NULL, dict(out=None)),
    (ARG, dict(experts=1025, ld=2048, ldo=2048)), (ARG, dict(topk=65)), (ARG, dict(experts=1, topk=2)), (ARG, dict(ld=10)),
    (ARG, dict(ldo=10)), (ARG, dict(tokens=1 << 22)), (DTYPE, dict(dt=I8)), (ALIGN, dict(out=F + 1)), (ALIGN, dict(dw=F + 2)),
    (ALIGN, dict(dl=F + 1)), (ALIGN, dict(counts=F + 2)), (OK, dict(tokens=0)),
])
def test_route_backward_refusals(want, kw):
    assert route_backward(**kw) == want


def quant4(x=F, ld=64, rows=4, k=64, dt=BF16, group=32, codes=F, ldc=32, scales=F):
    return rx.lib().rx_quant_fp4(x, ld, rows, k, dt, group, codes, ldc, scales, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(codes=None)), (NULL, dict(scales=None)), (ARG, dict(group=16)), (ARG, dict(group=0)),
    (ARG, dict(group=-32)), (ARG, dict(group=256)), (ARG, dict(rows=1 << 22)), (ARG, dict(ld=63)), (ARG, dict(ldc=31)),
    (ARG, dict(k=(1 << 23) + 1, ld=1 << 24, ldc=1 << 24)), (DTYPE, dict(dt=rx.RX_FP8_E4M3)), (ALIGN, dict(x=F + 1)),
    (ALIGN, dict(scales=F + 2)), (OK, dict(rows=0)), (OK, dict(k=0)),
])
def test_quant_fp4_refusals(want, kw):
    assert quant4(**kw) == want


def gemm4(a=F, lda=64, b=F, ldb=32, stride=0, scales=F, group=32, offsets=None, experts=1, rows=4, n=8, k=64, dt=BF16, out=F, ldo=8):
    return rx.lib().rx_gemm_fp4(a, lda, b, ldb, stride, scales, group, offsets, experts, rows, n, k, dt, out, ldo, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(a=None)), (NULL, dict(b=None)), (NULL, dict(scales=None)), (NULL, dict(out=None)), (ARG, dict(group=48)),
    (ARG, dict(experts=0)), (ARG, dict(experts=2)), (ARG, dict(offsets=F, experts=1025)), (ARG, dict(lda=63)), (ARG, dict(ldo=7)),
    (ARG, dict(ldb=16)), (ARG, dict(k=65)), (ARG, dict(rows=1 << 22)), (ARG, dict(n=1 << 31, ldo=1 << 31)), (ARG, dict(lda=1 << 23)),
    (ARG, dict(ldb=1 << 23)), (ARG, dict(k=(1 << 23) + 1, lda=1 << 24, ldb=1 << 24)),
    (ARG, dict(rows=(1 << 22) - 1, n=1 << 14, ldo=1 << 14)), (DTYPE, dict(dt=I8)), (ALIGN, dict(a=F + 1)), (ALIGN, dict(b=F + 8)),
    (ALIGN, dict(ldb=40)), (ALIGN, dict(stride=8, offsets=F)), (ALIGN, dict(scales=F + 2)), (ALIGN, dict(offsets=F + 2)),
    (ALIGN, dict(dt=FP32, out=F + 2)), (OK, dict(rows=0)), (OK, dict(n=0)),
])
def test_gemm_fp4_refusals(want, kw):
    assert gemm4(**kw) == want


def layer_norm(srcs=(F, F), lds=64, bias=None, res=None, ldr=64, w=F, b=F, eps=1e-5, drop=0.0, rng=None, rows=4, hidden=64, dt=BF16, h=F,
               ldh=64, z=F, ldz=64, mean=None, rstd=None, nsrc=None):
    return rx.lib().rx_layer_norm(None if srcs is None else ptrs(*srcs), len(srcs or ()) if nsrc is None else nsrc, lds, bias, res, ldr, w, b,
                                  eps, drop, rng, rows, hidden, dt, h, ldh, z, ldz, mean, rstd, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(srcs=None)), (NULL, dict(srcs=(F, None))), (NULL, dict(h=None, z=None)), (NULL, dict(drop=0.5)),
    (ARG, dict(nsrc=0)), (ARG, dict(nsrc=17)), (ARG, dict(eps=0.0)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=NAN)), (ARG, dict(eps=float("inf"))),
    (ARG, dict(drop=-0.1, rng=F)), (ARG, dict(drop=1.0, rng=F)), (ARG, dict(drop=NAN, rng=F)), (ARG, dict(drop=0.999999, rng=F)),
    (ARG, dict(hidden=32769, lds=32769, ldh=32769, ldz=32769)), (ARG, dict(rows=1 << 22)), (ARG, dict(lds=63)), (ARG, dict(ldh=63)),
    (ARG, dict(ldz=1)), (ARG, dict(res=F, ldr=63)), (DTYPE, dict(dt=I8)), (ALIGN, dict(srcs=(F, F + 1))), (ALIGN, dict(bias=F + 1)),
    (ALIGN, dict(w=F + 1)), (ALIGN, dict(z=F + 1)), (ALIGN, dict(mean=F + 2)), (ALIGN, dict(drop=0.5, rng=F + 4)),
    (OK, dict(rows=0)), (OK, dict(hidden=0)), (OK, dict(rows=0, h=None, z=None, srcs=(None,))),
])
def test_layer_norm_refusals(want, kw):
    assert layer_norm(**kw) == want


def layer_norm_backward(h=F, ldh=64, w=F, mean=F, rstd=F, drop=0.0, rng=None, rows=4, hidden=64, dt=BF16, dh=F, lddh=64, dz=F, lddz=64, ds=F,
                        ldds=64, dr=None, lddr=64, dbias=None, dw=None, db=None, ws=F, wsb=1 << 30):
    return rx.lib().rx_layer_norm_backward(h, ldh, w, mean, rstd, drop, rng, rows, hidden, dt, dh, lddh, dz, lddz, ds, ldds, dr, lddr, dbias,
                                           dw, db, ws, wsb, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(h=None)), (NULL, dict(mean=None)), (NULL, dict(rstd=None)), (NULL, dict(drop=0.25)), (ARG, dict(drop=1.5, rng=F)),
    (ARG, dict(rows=1 << 22)), (ARG, dict(hidden=40000, ldh=40000, lddh=40000, lddz=40000, ldds=40000)), (ARG, dict(ldh=63)),
    (ARG, dict(lddh=63)), (ARG, dict(lddz=63)), (ARG, dict(ldds=63)), (ARG, dict(dr=F + 64, lddr=63)), (ARG, dict(dr=F)), (DTYPE, dict(dt=I8)),
    (ALIGN, dict(dz=F + 1)), (ALIGN, dict(dw=F + 2)), (ALIGN, dict(drop=0.5, rng=F + 4)), (OK, dict(rows=0)), (OK, dict(hidden=0, dw=F)),
])
def test_layer_norm_backward_refusals(want, kw):
    assert layer_norm_backward(**kw) == want


def test_binding_refuses_cpu_tensors_and_what_is_no_matrix(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, i, u = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_moe_route(x, i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_moe_route_backward(x, i, torch.zeros(4), None, None, None, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_quant_fp4(x, u, torch.zeros(4, 1), 32)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_gemm_fp4(x, u, torch.zeros(4, 1), x, 32)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_layer_norm([x], None, None, None, x, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        rx.rx_layer_norm_backward(x, None, None, None, x, x, x)
    with pytest.raises(ValueError, match="two dimensions"):
        rx.rx_moe_route(torch.zeros(8), i, x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        rx.rx_moe_route(x.double(), i, x)
    with pytest.raises(ValueError, match="three dimensions"):
        rx.rx_gemm_fp4(x, u, x, x, 32, offsets=i)
    with pytest.raises(ValueError, match="group must be positive"):
        rx.rx_gemm_fp4(x, u, x, x, 0)
    with pytest.raises(ValueError, match="no gradient"):
        rx.rx_layer_norm_backward(None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="1 to 16 sources"):
        rx.rx_layer_norm([], None, None, None, x, None)


def test_reference_generator_against_the_published_numbers():
    """Known answers of Philox 4 x 32 with ten rounds, from its authors' distribution (kat_vectors)."""
    f = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = R.philox(np.array([counter], dtype=np.uint64), key)
        assert tuple(int(v) for v in got[0]) == want


def test_reference_dropout_keeps_its_share():
    keep = R.kept(64, 1000, 0.3, torch.tensor([5, 7]))
    # 64000 independent draws: five standard deviations of 0.0018
    assert abs(keep.double().mean().item() - (1 - R.threshold(0.3) / 65536)) < 0.0091


@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_route_gradient_against_differences(renormalize):
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    t, e, k = 6, 7, 3
    x = rnd(t, e)
    x[1, 2:] = -torch.inf
    x[2] = -torch.inf
    mask = torch.tensor([1, 1, 1, 0, 1, 1])
    B.HALF[torch.float64] = 0.0
    f = R.route(x, mask, k, renormalize)
    dw, dl = rnd(t, k), rnd(2)
    d, _ = R.route_backward(x, f, dw, dl, renormalize)
    assert bool((d[2] == 0).all()) and bool((d[3] == 0).all())
    step = 1e-5
    dirn = rnd(t, e)
    vals = []
    for sign in (1, -1):
        y = torch.where(torch.isinf(x), x, x + sign * step * dirn)
        o = R.route(y, mask, k, renormalize)
        assert torch.equal(o["ids"], f["ids"])
        vals.append(((o["weights"][0] * dw).sum() + (o["losses"][0] * dl).sum()).item())
    want = (vals[0] - vals[1]) / (2 * step)
    # truncation step^2 times third derivatives of order 100, rounding 1e-16 * 100 / step
    assert abs(want - (d * torch.where(torch.isinf(x), 0.0, dirn)).sum().item()) < 1e-7 * max(1.0, abs(want))


@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_reference_layer_norm_gradient_against_differences(drop):
    g = torch.Generator().manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    rows, n, eps = 4, 11, 1e-3
    rng = torch.tensor([11, 13])
    t = dict(src=rnd(rows, n), residual=rnd(rows, n), bias=rnd(n), w=rnd(n), b=rnd(n))
    other, dh, dz = rnd(rows, n), rnd(rows, n), rnd(rows, n)
    B.HALF[torch.float64] = 0.0

    def forward(t):
        h, _ = R.block_end([t["src"], other], t["bias"], t["residual"], drop, rng)
        return h, R.layer_norm(h, t["w"], t["b"], eps)

    h, f = forward(t)
    grads = R.layer_norm_backward(h, t["w"], f["mean"][0], f["rstd"][0], dh, dz, drop, rng)
    step = 1e-5
    for name in t:
        dirn = rnd(*t[name].shape)
        vals = []
        for sign in (1, -1):
            h1, f1 = forward(dict(t, **{name: t[name] + sign * step * dirn}))
            vals.append(((h1 * dh).sum() + (f1["z"][0] * dz).sum()).item())
        want = (vals[0] - vals[1]) / (2 * step)
        assert abs(want - (grads["d_" + name][0] * dirn).sum().item()) < 1e-7 * max(1.0, abs(want)), name


def test_reference_codes():
    """Ties to the even mantissa, the sign of a zero, and a group without values."""
    x = torch.tensor([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -0.0, 0.3]], dtype=torch.float32)
    code, s = R.quant_fp4(x, 32)
    assert s.tolist() == [[1.0]] and code.tolist() == [[7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 8, 1]]
    code, s = R.quant_fp4(torch.zeros(1, 3), 32)
    assert s.tolist() == [[1.0]] and code.tolist() == [[0, 0, 0]]
    assert R.pack4(torch.tensor([[1, 2, 3]], dtype=torch.uint8)).tolist() == [[0x21, 0x03]]
