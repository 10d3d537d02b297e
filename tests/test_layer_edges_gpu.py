"""The router and the layer norm at the edges of what their calls accept,
against their float64 forms (layer_ref.py) or plain arithmetic."""
import pytest
import torch

import allreduce_reduction_rx_amd as rx
import layer_ref as R
from block_ref import cast_bound
from test_block_ops_gpu import DTYPES, gen, randn, within
from test_layer_ops_gpu import F32, RNG

pytestmark = pytest.mark.gpu


# ---- layer norm: rows whose mean times 1 / sqrt(eps) is no float32 -------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("power,eps,hidden", [
    (120, 1e-5, 24), (120, 1e-5, 96),
    (110, 1e-12, 3), (110, 1e-12, 5), (110, 1e-12, 24), (110, 1e-12, 90), (110, 1e-12, 96), (110, 1e-12, 1001), (110, 1e-12, 1536),
    (110, 1e-12, 5001), (110, 1e-12, 8197)])
def test_layer_norm_gradient_of_large_equal_elements(power, eps, hidden, drop, dtype):
    """Elements of 2^power: sum, mean and the differences from it (zeros) are exact at these widths, the forward
    pass is finite, and so is the gradient, whichever lanes hold no element of the row."""
    g, rows, eps = gen(hidden), 37, torch.tensor(eps).item()   # eps: the float32 that the call gets
    res = torch.full((rows, hidden), 2.0 ** power).to(dtype)
    w, b = randn(g, hidden, dtype=dtype), randn(g, hidden, dtype=dtype)
    dh, dz = randn(g, rows, hidden, dtype=dtype), randn(g, rows, hidden, dtype=dtype)
    new = lambda *s, dtype=torch.float32: torch.full(s, 77.0, dtype=dtype, device="cuda")
    h, z, mu, rstd, rng = new(rows, hidden, dtype=dtype), new(rows, hidden, dtype=dtype), new(rows), new(rows), RNG.cuda() if drop else None
    rx.rx_layer_norm([torch.zeros(rows, hidden, dtype=dtype, device="cuda")], res.cuda(), w.cuda(), b.cuda(), h, z, mean=mu, rstd=rstd,
                     drop=drop, rng=rng, eps=eps)
    assert torch.equal(h.cpu(), res) and bool((mu == 2.0 ** power).all()) and torch.equal(z.cpu(), b.expand(rows, hidden))
    ds, dr, sums = new(rows, hidden, dtype=dtype), new(rows, hidden, dtype=dtype), [new(hidden) for _ in range(3)]
    ws = torch.full((rx.rx_layer_norm_backward_workspace(rows, hidden),), 0xA5, dtype=torch.uint8, device="cuda")
    rx.rx_layer_norm_backward(h, w.cuda(), mu, rstd, dh.cuda(), dz.cuda(), ds, d_residual=dr, d_bias=sums[0], d_w=sums[1], d_b=sums[2],
                              drop=drop, rng=rng, workspace=ws)
    want = R.layer_norm_backward(res, w, mu.cpu(), rstd.cpu(), dh, dz, drop, RNG)
    for name, t in (("d_src", ds), ("d_residual", dr)):
        within(t, want[name][0], cast_bound(*want[name], dtype))
    for name, t in (("d_bias", sums[0]), ("d_w", sums[1]), ("d_b", sums[2])):
        within(t, *want[name])


# ---- router: gradients that are NaN ---------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,topk", [(5, 2), (64, 8), (160, 6), (1000, 3)])
def test_route_gradient_of_every_nan(experts, topk, renormalize, dtype):
    """A NaN of a choice's gradient makes its token's gradient NaN, whatever the NaN's bits: of every element, with
    renormalize of the chosen ones. The other tokens' stay as they are."""
    bits = [0x7FFFDEAD, 0x7FC00000, 0x7F800001, 0x7FFFFFFF, -1, 0xFF800001 - (1 << 32)]
    g, tokens = gen(experts), 2 * len(bits) + 1
    x = randn(g, tokens, experts).to(dtype).cuda()
    ids, weights, lse = torch.empty(tokens, topk, dtype=torch.int32, device="cuda"), torch.empty(tokens, topk, **F32), torch.empty(tokens, **F32)
    rx.rx_moe_route(x, ids, weights, renormalize=renormalize, lse=lse)
    dw = randn(g, tokens, topk).cuda()
    clean, d = torch.empty_like(x), torch.empty_like(x)
    rx.rx_moe_route_backward(x, ids, lse, None, dw, None, clean, renormalize=renormalize)
    assert bool(clean.isfinite().all())
    at = torch.arange(1, 2 * len(bits), 2, device="cuda")
    dw.view(torch.int32)[at, at % topk] = torch.tensor(bits, dtype=torch.int32, device="cuda")
    assert int(dw.isnan().sum()) == len(bits)
    rx.rx_moe_route_backward(x, ids, lse, None, dw, None, d, renormalize=renormalize)
    bad = torch.zeros(tokens, experts, dtype=torch.bool, device="cuda")
    if renormalize:
        bad[at[:, None], ids[at].long()] = True
    else:
        bad[at] = True
    assert torch.equal(d.isnan(), bad)
    others = torch.arange(0, tokens, 2, device="cuda")
    assert torch.equal(d[others], clean[others])
