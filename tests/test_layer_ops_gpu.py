"""The router, the products with 4-bit weights and the layer norm on the GPU
against their float64 forms (layer_ref.py, whose bounds are counted from the
roundings)."""
import pytest
import torch

import allreduce_reduction_rx_amd as rx
import layer_ref as R
from block_ref import HALF, cast_bound
from test_block_ops_gpu import BF16, DTYPES, FP32, Strided, gen, gpu, put, randn, within

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
F32 = dict(dtype=torch.float32, device="cuda")


def inside(got, pair):
    """As within(), where infinities and NaN have to be the same."""
    want, bound = pair
    got = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)) and torch.equal(got[~fine].nan_to_num(5), want[~fine].nan_to_num(5))
    within(torch.where(fine, got, 0.0), torch.where(fine, want, 0.0), torch.where(fine, bound, 0.0))


# ---- router ------------------------------------------------------------------------

def run_route(logits, mask, topk, renormalize, sums=True, stream=None):
    t, e = logits.shape
    ids, weights = torch.full((t, topk), -77, **I32), torch.full((t, topk), 77.0, **F32)
    lse = torch.full((t,), 77.0, **F32)
    counts, losses = (torch.full((e + 1,), -77, **I32), torch.full((2,), 77.0, **F32)) if sums else (None, None)
    ws = torch.full((rx.rx_moe_route_workspace(t, e),), 0xA5, dtype=torch.uint8, device="cuda") if sums else None
    rx.rx_moe_route(logits, ids, weights, token_mask=mask, renormalize=renormalize, lse=lse, counts=counts, losses=losses,
                    workspace=ws, stream=stream)
    return ids, weights, lse, counts, losses


def check_route(x, mask, topk, renormalize, strided=False):
    t, e = x.shape
    xg = put(Strided(t, e, x.dtype, extra=3), x) if strided else x.cuda()
    mg = gpu(mask)
    f = R.route(x, mask, topk, renormalize)
    ids, weights, lse, counts, losses = run_route(xg, mg, topk, renormalize)
    torch.cuda.synchronize()
    assert torch.equal(ids.cpu(), f["ids"])
    assert torch.equal(counts.cpu(), f["counts"])
    inside(weights, f["weights"])
    inside(lse, f["lse"])
    inside(losses, f["losses"])
    bare = run_route(xg, mg, topk, renormalize, sums=False)
    assert torch.equal(bare[0], ids) and torch.equal(bare[1], weights) and torch.equal(bare[2], lse)
    g = gen(t)
    dw, dl = randn(g, t, topk), randn(g, 2) * max(1, t)
    for a, b in ((dw, dl), (dw, None), (None, dl), (None, None)):
        guard = Strided(t, e, x.dtype)
        rx.rx_moe_route_backward(xg, ids, lse, counts if b is not None else None, gpu(a), gpu(b), guard.t, renormalize=renormalize)
        torch.cuda.synchronize()
        guard.check()
        within(guard.t, *R.route_backward(x, f, a, b, renormalize))


def logits_of(g, tokens, experts, dtype, closed=0, empty=0):
    x = randn(g, tokens, experts, scale=2.0)
    if closed:
        x[:, torch.randperm(experts, generator=g)[:closed]] = -torch.inf
    x = x.to(dtype)
    x[:empty] = -torch.inf
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("tokens,experts,topk,closed,empty", [
    (1, 1, 1, 0, 0), (1, 64, 8, 0, 0), (3, 5, 5, 2, 1), (65, 8, 2, 0, 0), (70, 7, 7, 0, 0), (33, 16, 4, 10, 2), (17, 24, 3, 0, 0),
    (129, 64, 64, 0, 3), (130, 100, 6, 99, 0), (40, 128, 8, 0, 0), (9, 160, 6, 20, 0), (31, 257, 9, 0, 1), (12, 512, 16, 500, 0),
    (10, 1000, 64, 0, 0), (5, 1024, 3, 0, 1), (3000, 40, 4, 0, 0)])
def test_route(dtype, renormalize, tokens, experts, topk, closed, empty):
    g = gen(tokens * 1000 + experts)
    x = logits_of(g, tokens, experts, dtype, closed, empty)
    mask = torch.rand(tokens, generator=g) < 0.9 if tokens > 2 else None
    check_route(x, mask, topk, renormalize, strided=tokens % 2 == 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_of_many_tokens(dtype):
    """More tokens than one round of all workgroups has."""
    check_route(logits_of(gen(1), 40001, 20, dtype), None, 4, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,topk", [(8, 8), (48, 5), (1024, 20)])
def test_route_ties_go_to_the_lowest_number(dtype, experts, topk):
    g = gen(experts)
    x = torch.randint(-1, 2, (50, experts), generator=g).to(dtype)
    x[:5] = 0.0
    x[:5, ::2] = -0.0   # equals 0
    check_route(x, None, topk, False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_far_logits(dtype):
    """Of a type's whole range: exp underflows to 0, lse is the largest."""
    x = torch.tensor([[3e38, 1.0, -3e38, 0.0], [-3e38, -3e38, -3e38, -torch.inf], [200.0, 100.0, 0.0, -100.0], [1e-38, 0, 0, 0]]).to(dtype)
    f = R.route(x, None, 3, True)
    ids, weights, lse, counts, _ = run_route(x.cuda(), None, 3, True)
    assert torch.equal(ids.cpu(), f["ids"]) and torch.equal(counts.cpu(), f["counts"])
    inside(weights, f["weights"])
    inside(lse, f["lse"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_nan_stays_with_its_token(dtype):
    x = logits_of(gen(3), 40, 12, dtype)
    clean = run_route(x.cuda(), None, 3, False)
    bad = x.clone()
    bad[7, 4] = torch.nan
    bad[9, 2], bad[9, 3] = -torch.nan, torch.inf
    mask = torch.ones(40, dtype=torch.uint8)
    ids, weights, lse, counts, losses = run_route(bad.cuda(), mask.cuda(), 3, False)
    assert bool(((ids >= 0) & (ids < 12)).all()) and ids[7, 0] == 4 and ids[9, 0] == 2
    assert bool(weights[[7, 9]].isnan().all()) and bool(losses.isnan().all())
    others = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(ids[others], clean[0][others]) and torch.equal(weights[others], clean[1][others])
    mask[[7, 9]] = 0   # left out, they are not looked at
    ids, weights, lse, counts, losses = run_route(bad.cuda(), mask.cuda(), 3, False)
    f = R.route(x, mask, 3, False)
    assert torch.equal(ids.cpu(), f["ids"])
    inside(losses, f["losses"])
    d = torch.full((40, 12), 7.0, dtype=dtype, device="cuda")
    rx.rx_moe_route_backward(bad.cuda(), ids, lse, counts, torch.ones(40, 3, **F32), torch.ones(2, **F32), d)
    assert bool((d[[7, 9]] == 0).all()) and bool(d.isfinite().all())


def test_route_without_tokens():
    for mask, tokens in ((None, 0), (torch.zeros(9, dtype=torch.bool), 9)):
        x = torch.randn(tokens, 6).cuda()
        ids, weights, lse, counts, losses = run_route(x, gpu(mask), 2, True)
        assert counts.tolist() == [0] * 7 and losses.tolist() == [0.0, 0.0]
        assert bool((ids == -1).all()) and bool((weights == 0).all()) and bool((lse == -torch.inf).all())
        d = torch.full((tokens, 6), 7.0, device="cuda")
        rx.rx_moe_route_backward(x, ids, lse, counts, weights, losses, d)
        assert bool((d == 0).all())


@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_in_place_and_with_the_counts_of_several_ranks(renormalize):
    g = gen(8)
    xs = [randn(g, 30, 10) for _ in range(2)]
    outs = [run_route(x.cuda(), None, 3, renormalize) for x in xs]
    counts = outs[0][3] + outs[1][3]
    both = R.route(torch.cat(xs), None, 3, renormalize)
    assert torch.equal(counts.cpu(), both["counts"])
    dw, dl = randn(g, 60, 3), randn(g, 2) * 60
    want, bound = R.route_backward(torch.cat(xs), both, dw, dl, renormalize)
    for i in range(2):
        d = xs[i].cuda()
        rx.rx_moe_route_backward(d, outs[i][0], outs[i][2], counts, dw[30 * i:30 * i + 30].cuda(), dl.cuda(), d, renormalize=renormalize)
        within(d, want[30 * i:30 * i + 30], bound[30 * i:30 * i + 30])


def test_route_gradient_leaves_out_ids_that_are_no_expert():
    x = randn(gen(4), 20, 9)
    ids, _, lse, counts, _ = run_route(x.cuda(), None, 3, False)
    wild = ids.clone()
    wild[::2, 1] = 2 ** 31 - 1
    wild[1::2, 2] = -(2 ** 31)
    dw = randn(gen(5), 20, 3)
    d = torch.empty(20, 9, **F32)
    rx.rx_moe_route_backward(x.cuda(), wild, lse, None, dw.cuda(), None, d)
    f = R.route(x, None, 3, False)
    f["ids"] = torch.where((wild >= 0) & (wild < 9), wild, -1).cpu()
    within(d, *R.route_backward(x, f, dw, None, False))


# ---- 4-bit weights -------------------------------------------------------------------

def coded(w, group, pad=0, fill=0xFF):
    """Codes on the GPU, rows padded to 16 bytes and `pad` more, and scales, by the framework."""
    rows, k = w.shape
    half = (k + 1) // 2
    ld = (half + 15) // 16 * 16 + pad
    full = torch.full((rows, ld), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, -(-k // group)), 77.0, **F32)
    rx.rx_quant_fp4(w.cuda(), full[:, :half], scales, group)
    return full, full[:, :half], scales


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 2), (5, 31), (4, 32), (7, 33), (2, 127), (3, 129), (6, 1000), (2, 2056), (3, 4096), (1, 20001)])
def test_quant_fp4(dtype, group, rows, k):
    g = gen(rows * 100 + k)
    x = (randn(g, rows, k) * torch.exp(randn(g, rows, k))).to(dtype)
    x[0, :: 3] = 0
    if rows > 2:
        x[2] = 0
    full, codes, scales = coded(x, group, pad=16)
    code, s = R.quant_fp4(x, group)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(codes.cpu(), R.pack4(code))
    assert bool((full[:, (k + 1) // 2:] == 0xFF).all())
    strided = Strided(rows, k, dtype, extra=3)
    c2, s2 = torch.zeros_like(codes), torch.zeros_like(scales)
    rx.rx_quant_fp4(put(strided, x), c2, s2, group)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_quant_fp4_every_tie():
    """Values at and next to the borders between levels."""
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = torch.cat([borders, torch.nextafter(borders, torch.zeros(7)), torch.nextafter(borders, torch.full((7,), 9.0)), torch.tensor([6.0])])
    x = torch.cat([near, -near[:10]])[None]
    assert x.shape == (1, 32)
    _, codes, scales = coded(x, 32)
    code, s = R.quant_fp4(x, 32)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu(), R.pack4(code))


@pytest.mark.parametrize("dtype", DTYPES)
def test_quant_fp4_groups_that_are_not_finite(dtype):
    x = randn(gen(1), 4, 96).to(dtype)
    x[0, 40], x[1, 3], x[2, 70], x[2, 80] = torch.nan, torch.inf, -torch.inf, torch.nan
    _, codes, scales = coded(x, 32)
    assert bool(scales[0, 1].isnan()) and scales[1, 0] == torch.inf and bool(scales[2, 2].isnan())
    assert bool((codes[0, 16:32] == 0).all()) and bool((codes[1, :16] == 0).all()) and bool((codes[2, 32:48] == 0).all())
    ok = torch.isfinite(scales.cpu())
    assert torch.equal(scales.cpu()[ok], R.quant_fp4(torch.nan_to_num(x.float(), posinf=0, neginf=0).to(dtype), 32)[1][ok])
    out = torch.empty(1, 4, dtype=dtype, device="cuda")
    rx.rx_gemm_fp4(torch.ones(1, 96, dtype=dtype, device="cuda"), codes, scales, out, 32)
    assert out.isnan().tolist() == [[True, True, True, False]]


def some_codes(g, rows, k, group):
    """Codes of all levels, padded with whatever, and their scales of several sizes."""
    ld = (k + 31) // 32 * 16
    full = torch.randint(0, 256, (rows, ld), generator=g, dtype=torch.uint8)
    code = torch.stack([full & 15, full >> 4], 2).reshape(rows, -1)[:, :k]
    scales = torch.exp(randn(g, rows, -(-k // group)))
    return full, code, scales


def check_gemm(dtype, m, n, k, group, strided=False):
    g = gen(m + 10 * n + 100 * k)
    full, code, scales = some_codes(g, n, k, group)
    a = randn(g, m, k, dtype=dtype)
    guard = Strided(m, n, dtype)
    ag = put(Strided(m, k, dtype, extra=5), a) if strided else a.cuda()
    rx.rx_gemm_fp4(ag, full.cuda()[:, :(k + 1) // 2], scales.cuda(), guard.t, group)
    torch.cuda.synchronize()
    guard.check()
    within(guard.t, *R.gemm_fp4(a, code, scales, group))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k,group", [
    (1, 1, 1, 32), (1, 1, 2, 64), (1, 16, 32, 32), (2, 17, 33, 32), (1, 300, 128, 128), (3, 40, 127, 64), (16, 32, 129, 128), (17, 31, 96, 32),
    (5, 64, 1000, 64), (15, 100, 2056, 64), (32, 70, 257, 128), (33, 50, 512, 32), (64, 48, 640, 64), (65, 33, 200, 128), (100, 129, 333, 32),
    (130, 260, 1031, 128), (200, 300, 700, 64), (1, 8192, 1024, 128), (4, 2048, 4096, 32), (300, 520, 260, 32)])
def test_gemm_fp4_dense(dtype, m, n, k, group):
    check_gemm(dtype, m, n, k, group, strided=m % 2 == 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("m,n,k", [
    (1, 2000, 1304), (3, 5000, 2056), (13, 2000, 1304), (16, 5000, 2056), (16, 40000, 520), (20, 3000, 1304), (30, 5000, 1304), (30, 40000, 264),
    (60, 5000, 776), (61, 40000, 264), (600, 5000, 392), (1200, 9000, 136), (2000, 9000, 264)])
@pytest.mark.parametrize("odd", [0, 3])
def test_gemm_fp4_tiles(dtype, group, m, n, k, odd):
    """Sizes of every tile; rows of whole 16-byte units, and others."""
    check_gemm(dtype, m, n, k - odd, group)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,ks", [
    (3, 600, (900, 1024, 2048, 2056, 3100, 4100, 5128, 6200)), (13, 600, (900, 1024, 2048, 2056, 3100, 4100, 5128, 6200)),
    (16, 6000, (1000, 2048, 3100, 4104)), (30, 5000, (512, 520, 1100, 1600, 2100)), (60, 5000, (300, 512, 520, 1100, 1600, 2100)),
    (200, 6000, (8, 128, 136, 392, 520)), (2000, 9000, (8, 64, 128, 256, 640))])
def test_gemm_fp4_of_every_number_of_stages(dtype, m, n, ks):
    """k from one stage of a tile's buffers to more than there are of them, whole and partial."""
    for i, k in enumerate(ks):
        check_gemm(dtype, m, n, k, (32, 64, 128)[i % 3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,pad,n,k,group", [
    ([1], 0, 5, 40, 32), ([0, 3, 0, 1], 2, 20, 100, 64), ([4] * 16, 0, 40, 260, 128), ([20, 0, 33, 1, 70], 9, 130, 514, 32),
    ([0, 0], 4, 33, 64, 64), ([300, 5, 0, 129], 17, 70, 300, 64), ([1] * 70, 3, 33, 200, 128), ([2, 500], 1, 300, 129, 128),
    ([4] * 48, 5, 2500, 260, 64), ([3, 0, 5] * 16, 5, 2500, 264, 32)])
def test_gemm_fp4_grouped(dtype, counts, pad, n, k, group):
    g = gen(sum(counts) + n)
    experts, rows = len(counts), sum(counts) + pad
    parts = [some_codes(g, n, k, group) for _ in counts]
    offsets = torch.tensor([0] + counts).cumsum(0)
    a = randn(g, rows, k, dtype=dtype)
    guard = Strided(rows, n, dtype)
    rx.rx_gemm_fp4(a.cuda(), torch.stack([p[0] for p in parts]).cuda()[:, :, :(k + 1) // 2], torch.stack([p[2] for p in parts]).cuda(), guard.t,
                   group, offsets=offsets.int().cuda())
    torch.cuda.synchronize()
    guard.check()
    for e, (_, code, scales) in enumerate(parts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            within(guard.t[lo:hi], *R.gemm_fp4(a[lo:hi], code, scales, group))
    assert bool((guard.t[int(offsets[-1]):] == 0).all())


@pytest.mark.parametrize("m,n", [(3, 40), (200, 140)])
def test_gemm_fp4_rows_do_not_mix(m, n):
    """A NaN or an infinity stays in its row, and what lies behind k counts for nothing."""
    g = gen(2)
    k, group = 200, 64
    full, code, scales = some_codes(g, n, k, group)
    wide = randn(g, m, k + 24, dtype=BF16)
    wide[:, k:] = torch.nan
    a = wide[:, :k].clone()
    wide[1, 5] = torch.nan
    wide[2, 190] = torch.inf
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    rx.rx_gemm_fp4(wide.cuda()[:, :k], full.cuda()[:, :k // 2], scales.cuda(), out, group)
    rest = [i for i in range(m) if i not in (1, 2)]
    want, bound = R.gemm_fp4(a, code, scales, group)
    within(out[rest], want[rest], bound[rest])
    assert bool(out[1].isnan().all()) and not bool(out[2].isfinite().all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k,group", [(3, 40, 200, 64), (3, 20, 33, 32), (16, 5000, 520, 32), (200, 9000, 136, 32), (2000, 9000, 264, 64)])
def test_gemm_fp4_infinite_scales(dtype, m, n, k, group):
    """An infinite scale makes its channel infinite with its group's sign, also where a tile goes on behind k."""
    g = gen(k)
    full, code, scales = some_codes(g, n, k, group)
    code[5, :group], full[5, :group // 2] = 2, 0x22     # ones
    scales[5, 0] = torch.inf
    a = randn(g, m, k, dtype=dtype).abs() + 1
    out = torch.empty(m, n, dtype=dtype, device="cuda")
    rx.rx_gemm_fp4(a.cuda(), full.cuda()[:, :(k + 1) // 2], scales.cuda(), out, group)
    assert bool((out[:, 5] == torch.inf).all())
    scales[5, 0] = 1.0
    want, bound = R.gemm_fp4(a, code, scales, group)
    rest = [i for i in range(n) if i != 5]
    within(out[:, rest], want[:, rest], bound[:, rest])


@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemm_fp4_grouped_many_rows(group):
    """Large tiles that end inside an expert, an expert without rows and rows without an expert."""
    test_gemm_fp4_grouped(BF16, [700, 0, 1300, 129], 300, 4100, 264, group)
    test_gemm_fp4_grouped(torch.float32, [700, 0, 1300, 129], 300, 4100, 264, group)


def test_gemm_fp4_without_columns_or_rows():
    b, s = torch.zeros(40, 0, dtype=torch.uint8, device="cuda"), torch.zeros(40, 0, **F32)
    out = torch.full((3, 40), 7.0, **F32)
    rx.rx_gemm_fp4(torch.zeros(3, 0, **F32), b, s, out, 32)
    assert bool((out == 0).all())
    rx.rx_gemm_fp4(torch.zeros(0, 32, **F32), torch.zeros(40, 16, dtype=torch.uint8, device="cuda"), torch.zeros(40, 1, **F32), torch.zeros(0, 40, **F32), 32)


def test_gemm_fp4_offsets_outside_the_rows_are_clamped():
    g = gen(7)
    full, code, scales = some_codes(g, 24, 64, 32)
    a = randn(g, 6, 64, dtype=BF16)
    out = torch.zeros(6, 24, dtype=BF16, device="cuda")
    rx.rx_gemm_fp4(a.cuda(), full.cuda()[None].repeat(2, 1, 1), scales.cuda()[None].repeat(2, 1, 1), out, 32,
                   offsets=torch.tensor([-5, 2, 900], **I32))
    within(out, *R.gemm_fp4(a, code, scales, 32))


def test_gemm_fp4_exact_in_float32():
    """Small integers times levels: every partial sum is a float32 number, so each bit is known; 24 bits of a count."""
    g = gen(9)
    full, code, _ = some_codes(g, 40, 256, 32)
    scales = torch.ones(40, 8)
    a = torch.zeros(20, 256)
    a[torch.arange(20), torch.randint(0, 256, (20,), generator=g)] = 1 + torch.randint(0, 1 << 23, (20,), generator=g).float() * 2.0 ** -23
    out = torch.empty(20, 40, **F32)
    rx.rx_gemm_fp4(a.cuda(), full.cuda(), scales.cuda(), out, 32)
    want = a.double() @ R.values4(code).t()   # 24 bits times 1 or 3: up to 26 bits, one rounding
    assert torch.equal(out.cpu(), want.float())


# ---- layer norm ------------------------------------------------------------------------

RNG = torch.tensor([0x0123456789ABCDEF, -5])


def norm_run(rows, hidden, nsrc, dtype, drop=0.0, residual=True, bias=True, affine=True, strided=False, seed=0, mean=0.3):
    g = gen(seed + rows + hidden)
    mat = lambda t: put(Strided(rows, hidden, dtype), t) if strided else t.cuda()
    c = dict(srcs=[randn(g, rows, hidden, dtype=dtype) for _ in range(nsrc)], residual=(randn(g, rows, hidden) + mean).to(dtype) if residual else None,
             bias=randn(g, hidden, dtype=dtype) if bias else None, w=randn(g, hidden, dtype=dtype) if affine else None,
             b=randn(g, hidden, dtype=dtype) if affine else None, dh=randn(g, rows, hidden, dtype=dtype), dz=randn(g, rows, hidden, dtype=dtype))
    eps = 1e-5
    h, z = Strided(rows, hidden, dtype), Strided(rows, hidden, dtype)
    mu, rstd = torch.full((rows,), 77.0, **F32), torch.full((rows,), 77.0, **F32)
    rng = RNG.cuda() if drop else None
    rx.rx_layer_norm([mat(s) for s in c["srcs"]], None if c["residual"] is None else mat(c["residual"]), gpu(c["w"]), gpu(c["b"]), h.t, z.t,
                     bias=gpu(c["bias"]), mean=mu, rstd=rstd, drop=drop, rng=rng, eps=eps)
    torch.cuda.synchronize()
    h.check()
    z.check()
    want, bound = R.block_end(c["srcs"], c["bias"], c["residual"], drop, RNG)
    within(h.t, want, cast_bound(want, bound, dtype))
    hc = h.t.cpu()
    f = R.layer_norm(hc, c["w"], c["b"], eps)
    within(z.t, *f["z"])
    within(mu, *f["mean"])
    within(rstd, *f["rstd"])
    return c, h, mu, rstd, rng


def backward_run(c, h, mu, rstd, rng, drop, dtype, rows, hidden, dh=True, dz=True, strided=False):
    mat = lambda t: put(Strided(rows, hidden, dtype), t) if strided else t.cuda()
    ds, dr = Strided(rows, hidden, dtype), Strided(rows, hidden, dtype)
    sums = [torch.full((hidden,), 77.0, **F32) for _ in range(3)]
    ws = torch.full((rx.rx_layer_norm_backward_workspace(rows, hidden),), 0xA5, dtype=torch.uint8, device="cuda")
    rx.rx_layer_norm_backward(h.t, gpu(c["w"]), mu, rstd, mat(c["dh"]) if dh else None, mat(c["dz"]) if dz else None, ds.t, d_residual=dr.t,
                              d_bias=sums[0], d_w=sums[1], d_b=sums[2], drop=drop, rng=rng, workspace=ws)
    torch.cuda.synchronize()
    ds.check()
    dr.check()
    want = R.layer_norm_backward(h.t.cpu(), c["w"], mu.cpu(), rstd.cpu(), c["dh"] if dh else None, c["dz"] if dz else None, drop, RNG)
    for name, t in (("d_src", ds.t), ("d_residual", dr.t)):
        within(t, want[name][0], cast_bound(*want[name], dtype))
    for name, t in (("d_bias", sums[0]), ("d_w", sums[1]), ("d_b", sums[2])):
        within(t, *want[name])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("rows,hidden,nsrc", [
    (1, 1, 1), (2, 3, 2), (5, 8, 1), (3, 17, 16), (70, 64, 2), (33, 100, 3), (9, 512, 9), (300, 520, 1), (40, 1025, 2), (7, 2048, 4),
    (20, 4096, 2), (3, 5001, 3), (6, 8192, 8), (5, 8200, 2), (4, 10240, 1), (3, 16384, 2), (2, 20001, 2), (2, 32768, 1)])
def test_layer_norm_and_backward(dtype, drop, rows, hidden, nsrc):
    strided = rows % 2 == 1
    out = norm_run(rows, hidden, nsrc, dtype, drop, strided=strided)
    backward_run(*out, drop, dtype, rows, hidden, strided=strided)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,hidden", [(2000, 72), (1111, 1000), (700, 4096), (600, 8192), (520, 12000), (300, 16384)])
def test_layer_norm_of_many_rows(dtype, rows, hidden):
    """More rows than workgroups, at each width that has a kernel of its own."""
    out = norm_run(rows, hidden, 1, dtype, 0.1)
    backward_run(*out, 0.1, dtype, rows, hidden)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual,bias,affine,dh,dz", [
    (False, False, True, True, True), (True, False, False, False, True), (False, True, False, True, False), (True, True, True, False, False)])
def test_layer_norm_optional_operands(dtype, residual, bias, affine, dh, dz):
    for drop in (0.0, 0.5):
        out = norm_run(37, 200, 2, dtype, drop, residual, bias, affine)
        backward_run(*out, drop, dtype, 37, 200, dh, dz)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [40, 5000])
def test_layer_norm_outputs_are_optional(dtype, hidden):
    g = gen(hidden)
    rows = 12
    x, w, b, dz = (randn(g, *s, dtype=dtype).cuda() for s in ((rows, hidden), (hidden,), (hidden,), (rows, hidden)))
    z, mu, rstd = torch.empty_like(x), torch.empty(rows, **F32), torch.empty(rows, **F32)
    rx.rx_layer_norm([x], None, w, b, None, z, mean=mu, rstd=rstd)
    within(z, *R.layer_norm(x.cpu(), w.cpu(), b.cpu(), 1e-5)["z"])
    again = x.clone()
    rx.rx_layer_norm([again], None, w, b, None, again)   # in place
    assert torch.equal(again, z)
    h = torch.empty_like(x)
    rx.rx_layer_norm([x], None, None, None, h, None, drop=0.25, rng=RNG.cuda())
    keep = R.kept(rows, hidden, 0.25, RNG).cuda()
    assert torch.equal(h != 0, keep & (x != 0))
    ws = torch.empty(rx.rx_layer_norm_backward_workspace(rows, hidden), dtype=torch.uint8, device="cuda")
    full = torch.empty_like(x)
    rx.rx_layer_norm_backward(x, w, mu, rstd, None, dz, full, workspace=ws)
    dw = torch.empty(hidden, **F32)
    rx.rx_layer_norm_backward(x, w, mu, rstd, None, dz, None, d_w=dw, workspace=ws)   # the weight's alone
    within(dw, *R.layer_norm_backward(x.cpu(), w.cpu(), mu.cpu(), rstd.cpu(), None, dz.cpu(), 0.0, None)["d_w"])
    over = dz.clone()
    rx.rx_layer_norm_backward(x, w, mu, rstd, None, over, over, workspace=ws)   # over the gradient it came from
    assert torch.equal(over, full)
    # dropout's gradient alone: dH where it kept, as the forward call did
    d = torch.empty_like(x)
    rx.rx_layer_norm_backward(None, None, None, None, dz, None, d, drop=0.25, rng=RNG.cuda(), workspace=ws)
    assert torch.equal(d != 0, keep & (dz != 0))


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_in_place(dtype):
    rows, hidden = 30, 1031
    c, h, mu, rstd, rng = norm_run(rows, hidden, 2, dtype, 0.2)
    z = torch.empty(rows, hidden, dtype=dtype, device="cuda")
    for target in range(3):
        srcs, res = [gpu(s) for s in c["srcs"]], gpu(c["residual"])
        out = (srcs + [res])[target]
        rx.rx_layer_norm(srcs, res, gpu(c["w"]), gpu(c["b"]), out, z, bias=gpu(c["bias"]), drop=0.2, rng=rng)
        assert torch.equal(out, h.t)
    ws = torch.empty(rx.rx_layer_norm_backward_workspace(rows, hidden), dtype=torch.uint8, device="cuda")
    ds, dr = torch.empty_like(z), torch.empty_like(z)
    call = lambda dh, dz, s, r: rx.rx_layer_norm_backward(h.t, gpu(c["w"]), mu, rstd, dh, dz, s, d_residual=r, drop=0.2, rng=rng, workspace=ws)
    call(gpu(c["dh"]), gpu(c["dz"]), ds, dr)
    a, b = gpu(c["dh"]), gpu(c["dz"])
    call(a, b, b, a)
    assert torch.equal(a, dr) and torch.equal(b, ds)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropped_elements_are_zero_whatever_they_were(dtype):
    rows, hidden = 6, 77
    keep = R.kept(rows, hidden, 0.5, RNG)
    x = randn(gen(1), rows, hidden, dtype=dtype)
    bad = torch.where(keep, x, torch.tensor(torch.nan, dtype=dtype))
    bad[0] = torch.where(keep[0], x[0], torch.tensor(torch.inf, dtype=dtype))
    h, want = torch.empty(rows, hidden, dtype=dtype, device="cuda"), torch.empty(rows, hidden, dtype=dtype, device="cuda")
    z = torch.empty_like(h)
    rx.rx_layer_norm([x.cuda()], None, None, None, want, z, drop=0.5, rng=RNG.cuda())
    rx.rx_layer_norm([bad.cuda()], None, None, None, h, z, drop=0.5, rng=RNG.cuda())
    assert torch.equal(h, want) and bool(h.isfinite().all())


@pytest.mark.parametrize("seed,offset", [(0, 0), (-1, -1), (1 << 62, 3), (7, 1 << 40), (-(1 << 63), (1 << 63) - 1)])
def test_dropout_of_every_seed_and_offset(seed, offset):
    rng = torch.tensor([seed, offset])
    for dtype, hidden in ((BF16, 50), (FP32, 44), (FP32, 13)):
        x = torch.ones(20, hidden, dtype=dtype, device="cuda")
        h = torch.empty_like(x)
        rx.rx_layer_norm([x], None, None, None, h, None, drop=0.37, rng=rng.cuda())
        keep = R.kept(20, hidden, 0.37, rng)
        want = torch.where(keep, 65536 / (65536 - R.threshold(0.37)), 0.0).to(torch.float32).to(dtype)
        assert torch.equal(h.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [0.0, 1.0, 300.0, 1e15])
def test_layer_norm_of_rows_without_spread(value, dtype):
    """Equal elements: the variance is 0 but for the mean's rounding, rstd 1 / sqrt(eps) at the most."""
    x = torch.full((3, 1500), value, dtype=dtype, device="cuda")
    z, mu, rstd = torch.empty_like(x), torch.empty(3, **F32), torch.empty(3, **F32)
    rx.rx_layer_norm([x], None, None, None, None, z, mean=mu, rstd=rstd)
    f = R.layer_norm(x.cpu(), None, None, 1e-5)
    within(mu, *f["mean"])
    assert bool(torch.isfinite(z).all()) and bool((rstd <= 1 / 1e-5 ** 0.5 * (1 + 2 ** -20)).all())
    if value in (0.0, 1.0):   # sums of ones are exact up to 2^24; the mean then rounds twice
        within(z, *f["z"])


def test_layer_norm_without_rows():
    x = torch.empty(0, 24, **F32)
    rx.rx_layer_norm([x], None, None, None, x, x)
    ws = torch.empty(max(16, rx.rx_layer_norm_backward_workspace(0, 24)), dtype=torch.uint8, device="cuda")
    sums = [torch.full((24,), 7.0, **F32) for _ in range(3)]
    rx.rx_layer_norm_backward(x, None, torch.empty(0, **F32), torch.empty(0, **F32), x, x, x, d_bias=sums[0], d_w=sums[1], d_b=sums[2], workspace=ws)
    assert all(bool((s == 0).all()) for s in sums)


# ---- refusals, far offsets, streams, graphs -----------------------------------------------

def test_layer_binding_refusals():
    z = lambda *s, dtype=FP32: torch.zeros(*s, dtype=dtype, device="cuda")
    i, u = z(4, 2, dtype=torch.int32), z(8, 16, dtype=torch.uint8)
    refused = [
        (ValueError, "shape", lambda: rx.rx_moe_route(z(4, 8), i, z(4, 3))),
        (TypeError, "Int", lambda: rx.rx_moe_route(z(4, 8), i.long(), z(4, 2))),
        (ValueError, "shape", lambda: rx.rx_moe_route(z(4, 8), i, z(4, 2), token_mask=z(5, dtype=torch.bool))),
        (TypeError, "Bool", lambda: rx.rx_moe_route(z(4, 8), i, z(4, 2), token_mask=z(4))),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_moe_route(z(4, 8), i, z(4, 2), counts=z(9, dtype=torch.int32))),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_moe_route(z(4, 8), i, z(4, 2), counts=z(9, dtype=torch.int32), losses=z(2))),
        (rx.RxError, "RX_ERR_ARG", lambda: rx.rx_moe_route(z(4, 1), i, z(4, 2))),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_moe_route_backward(z(4, 8), i, z(4), None, None, z(2), z(4, 8))),
        (ValueError, "shape", lambda: rx.rx_quant_fp4(z(8, 33), u, z(8, 2), 32)),
        (rx.RxError, "RX_ERR_ARG", lambda: rx.rx_quant_fp4(z(8, 32), u, z(8, 2), 16)),
        (ValueError, "shape", lambda: rx.rx_gemm_fp4(z(4, 32), u, z(8, 2), z(4, 8), 32)),
        (ValueError, "padded", lambda: rx.rx_gemm_fp4(z(4, 24), torch.as_strided(z(7 * 16 + 12, dtype=torch.uint8), (8, 12), (16, 1)), z(8, 1), z(4, 8), 32)),
        (rx.RxError, "RX_ERR_ALIGN", lambda: rx.rx_gemm_fp4(z(4, 32), z(8, 24, dtype=torch.uint8)[:, :16], z(8, 1), z(4, 8), 32)),
        (ValueError, "another row stride", lambda: rx.rx_layer_norm([z(4, 8), z(4, 9)[:, :8]], None, None, None, z(4, 8), None)),
        (ValueError, "shape", lambda: rx.rx_layer_norm([z(4, 8)], None, z(9), None, None, z(4, 8))),
        (TypeError, "Float", lambda: rx.rx_layer_norm([z(4, 8)], None, z(8, dtype=BF16), None, None, z(4, 8))),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_layer_norm([z(4, 8)], None, None, None, None, None)),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_layer_norm([z(4, 8)], None, None, None, z(4, 8), None, drop=0.5)),
        (TypeError, "Long", lambda: rx.rx_layer_norm([z(4, 8)], None, None, None, z(4, 8), None, drop=0.5, rng=z(2))),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_layer_norm_backward(z(4, 8), None, z(4), z(4), None, z(4, 8), z(4, 8))),
        (rx.RxError, "RX_ERR_NULL", lambda: rx.rx_layer_norm_backward(None, None, None, None, None, z(4, 8), z(4, 8), workspace=z(4096, dtype=torch.uint8))),
    ]
    for error, match, call in refused:
        with pytest.raises(error, match=match):
            call()


def test_layer_row_offsets_past_32_bits():
    ld = (1 << 31) + 64
    g = gen(6)
    big = torch.empty(3 * ld, dtype=BF16, device="cuda")
    far = torch.as_strided(big, (3, 64), (ld, 1), 0)
    x = randn(g, 3, 64, dtype=BF16)
    far.copy_(x)
    f = R.route(x, None, 4, True)
    ids, weights, lse, counts, _ = run_route(far, None, 4, True)
    assert torch.equal(ids.cpu(), f["ids"])
    z, mu, rstd = torch.empty(3, 64, dtype=BF16, device="cuda"), torch.empty(3, **F32), torch.empty(3, **F32)
    rx.rx_layer_norm([far], None, None, None, None, z, mean=mu, rstd=rstd)
    within(z, *R.layer_norm(x, None, None, 1e-5)["z"])
    ws = torch.empty(rx.rx_layer_norm_backward_workspace(3, 64), dtype=torch.uint8, device="cuda")
    d = torch.empty_like(z)
    rx.rx_layer_norm_backward(far, None, mu, rstd, None, far, d, workspace=ws)
    want = R.layer_norm_backward(x, None, mu.cpu(), rstd.cpu(), None, x, 0.0, None)["d_src"]
    within(d, want[0], cast_bound(*want, BF16))
    dw = randn(g, 3, 4)
    dl = torch.empty(3, 64, dtype=BF16, device="cuda")
    rx.rx_moe_route_backward(far, ids, lse, None, dw.cuda(), None, dl, renormalize=True)
    within(dl, *R.route_backward(x, f, dw, None, True))
    parts = [some_codes(g, 16, 64, 32) for _ in range(2)]
    w = torch.as_strided(big.view(torch.uint8), (2, 16, 32), (2 * ld, 32, 1), 0)
    w.copy_(torch.stack([p[0] for p in parts]))
    a = randn(g, 4, 64, dtype=BF16)
    o = torch.empty(4, 16, dtype=BF16, device="cuda")
    rx.rx_gemm_fp4(a.cuda(), w, torch.stack([p[2] for p in parts]).cuda(), o, 32, offsets=torch.tensor([0, 1, 4], **I32))
    within(o[:1], *R.gemm_fp4(a[:1], parts[0][1], parts[0][2], 32))
    within(o[1:], *R.gemm_fp4(a[1:], parts[1][1], parts[1][2], 32))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(2000, 9000, 264), (13, 40, 200)])
def test_gemm_fp4_with_the_widest_row_stride(dtype, m, n, k):
    """Rows as far apart as they may be: 34 and 67 GB of them, tiles whose own rows span 2^31 bytes."""
    g = gen(12)
    full, code, scales = some_codes(g, n, k, 64)
    a = randn(g, m, k, dtype=dtype)
    ld = (1 << 23) - 8
    far = torch.as_strided(torch.empty((m - 1) * ld + k, dtype=dtype, device="cuda"), (m, k), (ld, 1))
    far.copy_(a)
    out = torch.empty(m, n, dtype=dtype, device="cuda")
    rx.rx_gemm_fp4(far, full.cuda()[:, :(k + 1) // 2], scales.cuda(), out, 64)
    within(out, *R.gemm_fp4(a, code, scales, 64))


class Block:
    """Buffers of one pass: route, dispatch, 4-bit products, combine, the block's end, and the gradients."""

    def __init__(self, seed, tokens=48, topk=3, experts=6, hidden=136):
        g = gen(seed)
        self.x, self.res, self.dh, self.dz = (randn(g, tokens, hidden, dtype=BF16).cuda() for _ in range(4))
        self.logits = randn(g, tokens, experts).cuda()
        self.mask = (torch.rand(tokens, generator=g) < 0.9).cuda()
        self.w_full, _, s = some_codes(g, experts * hidden, hidden, 32)
        self.w = self.w_full.cuda().view(experts, hidden, -1)[:, :, :hidden // 2]
        self.s = (0.05 * s).cuda().view(experts, hidden, -1)
        self.nw, self.nb, self.bias = (randn(g, hidden, dtype=BF16).cuda() for _ in range(3))
        self.rng = torch.tensor([seed, 99]).cuda()
        self.dl = torch.tensor([3.0, 0.5]).cuda()
        z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
        i = torch.int32
        pairs = tokens * topk
        self.ids, self.weights, self.lse, self.counts, self.losses = z(tokens, topk, dtype=i), z(tokens, topk, dtype=FP32), z(tokens, dtype=FP32), z(experts + 1, dtype=i), z(2, dtype=FP32)
        self.offsets, self.order, self.slots = z(experts + 1, dtype=i), z(pairs, dtype=i), z(tokens, topk, dtype=i)
        self.rows, self.y, self.out, self.h, self.z = z(pairs, hidden), z(pairs, hidden), z(tokens, hidden), z(tokens, hidden), z(tokens, hidden)
        self.mu, self.rstd = z(tokens, dtype=FP32), z(tokens, dtype=FP32)
        self.ds, self.dr, self.d_rows = z(tokens, hidden), z(tokens, hidden), z(pairs, hidden)
        self.sums = [z(hidden, dtype=FP32) for _ in range(3)]
        self.d_weights, self.d_logits = z(tokens, topk, dtype=FP32), z(tokens, experts, dtype=FP32)
        self.ws1 = z(rx.rx_moe_route_workspace(tokens, experts), dtype=torch.uint8)
        self.ws2 = z(rx.rx_layer_norm_backward_workspace(tokens, hidden), dtype=torch.uint8)
        self.experts = experts

    def run(self):
        rx.rx_moe_route(self.logits, self.ids, self.weights, token_mask=self.mask, renormalize=True, lse=self.lse, counts=self.counts,
                        losses=self.losses, workspace=self.ws1)
        rx.rx_moe_dispatch(self.ids, self.experts, self.offsets, self.order, self.slots, x=self.x, rows=self.rows)
        rx.rx_gemm_fp4(self.rows, self.w, self.s, self.y, 32, offsets=self.offsets)
        rx.rx_moe_combine(self.y, self.slots, self.weights, self.out)
        rx.rx_layer_norm([self.out], self.res, self.nw, self.nb, self.h, self.z, bias=self.bias, mean=self.mu, rstd=self.rstd, drop=0.2, rng=self.rng)
        rx.rx_layer_norm_backward(self.h, self.nw, self.mu, self.rstd, self.dh, self.dz, self.ds, d_residual=self.dr, d_bias=self.sums[0],
                                  d_w=self.sums[1], d_b=self.sums[2], drop=0.2, rng=self.rng, workspace=self.ws2)
        rx.rx_moe_combine_backward(self.ds, self.y, self.slots, self.weights, self.offsets, self.d_rows, self.d_weights)
        rx.rx_moe_route_backward(self.logits, self.ids, self.lse, self.counts, self.d_weights, self.dl, self.d_logits, renormalize=True)

    def buffers(self):
        return [self.ids, self.weights, self.lse, self.counts, self.losses, self.offsets, self.order, self.slots, self.rows, self.y, self.out, self.h,
                self.z, self.mu, self.rstd, self.ds, self.dr, self.d_rows, *self.sums, self.d_weights, self.d_logits]

    def results(self):
        return [t.clone() for t in self.buffers()]


def test_layers_together_on_another_stream_and_in_a_graph():
    b, other = Block(1), Block(2)
    b.run()
    torch.cuda.synchronize()
    want = b.results()
    # the counts are the dispatch's
    ends = b.offsets.tolist()
    assert [hi - lo for lo, hi in zip(ends, ends[1:])] == b.counts.tolist()[:-1]
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
    for i in range(4):
        for t in (*b.buffers(), b.ws1, b.ws2):
            t.fill_(1)
        other.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(b.results(), want))
    # the generator's numbers are read when the graph runs
    b.rng[1] += 1
    graph.replay()
    torch.cuda.synchronize()
    moved = b.results()
    b.run()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(moved, b.results()))
    assert not torch.equal(moved[11], want[11])
