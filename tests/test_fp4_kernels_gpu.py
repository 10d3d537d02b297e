"""The products with 4-bit weights, kernel by kernel: which one a call's sizes
select, and that each of them multiplies without loss, dense and by expert."""
import os
import subprocess
import sys

import pytest
import torch

import allreduce_reduction_rx_amd as rx
import layer_ref as R
from test_block_ops_gpu import BF16, FP32, Strided, gen, randn, within
from test_layer_ops_gpu import some_codes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"bf16": BF16, "fp32": FP32}

# type, rows, n, k, experts (0: dense), the kernel on 256 CUs. Rows of k that is no multiple of 8 go by way of registers.
KINDS = [
    ("fp32", 20, 40, 256, 0, "few"), ("fp32", 16, 5000, 520, 0, "stream 16x32"), ("fp32", 16, 9000, 301, 0, "stream 16x64"),
    ("fp32", 33, 30000, 259, 0, "stream 32x128"), ("fp32", 600, 5000, 391, 0, "parts"),
    ("fp32", 60, 200, 261, 12, "few"), ("fp32", 100, 1000, 264, 2, "stream 16x32"), ("fp32", 60, 2100, 264, 12, "stream 16x64"),
    ("fp32", 700, 2100, 263, 12, "stream 32x128"), ("fp32", 1500, 2100, 264, 12, "parts"),
    ("bf16", 3, 200, 1304, 0, "stream 16x16, four rows"), ("bf16", 3, 5000, 520, 0, "stream 16x32, four rows"),
    ("bf16", 13, 2000, 1304, 0, "stream 16x16"), ("bf16", 16, 5000, 520, 0, "stream 16x32"), ("bf16", 16, 20000, 520, 0, "stream 16x64"),
    ("bf16", 30, 5000, 264, 0, "stream 32x32"), ("bf16", 30, 40000, 264, 0, "stream 32x128"), ("bf16", 60, 5000, 264, 0, "stream 64x32"),
    ("bf16", 600, 5000, 392, 0, "stream 64x128"), ("bf16", 2000, 9000, 264, 0, "tile"),
    ("bf16", 60, 200, 264, 12, "stream 16x16"), ("bf16", 100, 1000, 264, 2, "stream 16x32"), ("bf16", 256, 2100, 264, 24, "stream 16x64"),
    ("bf16", 130, 1000, 264, 3, "stream 32x32"), ("bf16", 700, 2100, 264, 12, "stream 32x128"), ("bf16", 200, 1000, 264, 4, "stream 64x32"),
    ("bf16", 700, 2100, 264, 24, "stream 64x128"), ("bf16", 2500, 4100, 264, 4, "tile"),
    ("bf16", 100, 1000, 263, 2, "stream 16x32, rows by way of registers"), ("bf16", 256, 2100, 263, 24, "stream 16x64, rows by way of registers"),
    ("bf16", 130, 1000, 263, 3, "stream 32x32, rows by way of registers"), ("bf16", 700, 2100, 263, 12, "stream 32x128, rows by way of registers"),
    ("bf16", 200, 1000, 263, 4, "stream 64x32, rows by way of registers"), ("bf16", 700, 2100, 263, 24, "stream 64x128, rows by way of registers"),
]
NAMES = [f"{'dense' if not k[4] else 'experts'} {k[0]} {k[5]}" for k in KINDS]


def split(rows, experts):
    """Offsets of `experts`: rows dealt unevenly, one expert without any, and at last five rows that no expert has."""
    counts = [1 + (rows - 5 - experts) // experts + (i % 3 - 1) * (rows // (4 * experts)) for i in range(experts)]
    counts[1] = 0
    counts[0] += rows - 5 - sum(counts)
    return [0] + torch.tensor(counts).cumsum(0).tolist()


def one_each(g, rows, k, dtype):
    """Rows with one element that is not zero, at any place (the last one's among them), and its place. It has as
    many bits as a product with a level (1 or 3 times a power of two) leaves exact: 22 in FP32, the last of them
    set, so that none of the three parts of 8 bits is zero; 8 in BF16, before the result's rounding."""
    at = torch.randint(0, k, (rows,), generator=g)
    at[-1] = k - 1
    bits = 22 if dtype == FP32 else 8
    v = (1 << bits - 1) + 2 * torch.randint(0, 1 << bits - 2, (rows,), generator=g) + 1
    v = v.double() * 2.0 ** (1 - bits) * (1 - 2 * torch.randint(0, 2, (rows,), generator=g))
    a = torch.zeros(rows, k, dtype=torch.float64)
    a[torch.arange(rows), at] = v
    return a.to(dtype), v, at


def test_the_exact_rows_have_all_three_parts():
    a, v, at = one_each(gen(1), 50, 70, FP32)
    assert torch.equal(a.double()[torch.arange(50), at], v) and int((a != 0).sum()) == 50
    two = (a.view(torch.int32) & -0x100).view(torch.float32)   # the upper two parts
    assert bool((two != a).any(1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,m,n,k,experts,kernel", KINDS, ids=NAMES)
def test_products_are_exact(dtype, m, n, k, experts, kernel, group):
    """Products of 24 bits and scales that are powers of two: each bit is known; and sums of any numbers."""
    g = gen(m + n + k)
    dt = TYPES[dtype]
    parts = [some_codes(g, n, k, group) for _ in range(experts or 1)]
    for p in parts:
        p[2].copy_(torch.exp2(torch.randint(-3, 4, p[2].shape, generator=g).float()))
    ends = split(m, experts) if experts else [0, m]
    codes, scales = (torch.stack([p[i] for p in parts]).cuda() for i in (0, 2))
    codes = codes[:, :, :(k + 1) // 2]
    more = dict(offsets=torch.tensor(ends, dtype=torch.int32, device="cuda")) if experts else {}
    b, s = (codes, scales) if experts else (codes[0], scales[0])
    out = Strided(m, n, dt)
    a, v, at = one_each(g, m, k, dt)
    rx.rx_gemm_fp4(a.cuda(), b, s, out.t, group, **more)
    torch.cuda.synchronize()
    out.check()
    got = out.t.cpu()
    for e, (_, code, scale) in enumerate(parts):
        lo, hi = ends[e], ends[e + 1]
        w = R.values4(code[:, at[lo:hi]]) * scale[:, at[lo:hi] // group].double()
        assert torch.equal(got[lo:hi], (v[lo:hi] * w).t().to(FP32).to(dt))
    assert bool((got[ends[-1]:] == 0).all())
    a = randn(g, m, k, dtype=dt)
    rx.rx_gemm_fp4(a.cuda(), b, s, out.t, group, **more)
    torch.cuda.synchronize()
    out.check()
    for e, (_, code, scale) in enumerate(parts):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            within(out.t[lo:hi], *R.gemm_fp4(a[lo:hi], code, scale, group))
    assert bool((out.t[ends[-1]:] == 0).all())


CALLS = """
import sys, torch
import allreduce_reduction_rx_amd as rx
sys.path.insert(0, "tests")
from test_fp4_kernels_gpu import KINDS, TYPES, split
for i, (dtype, m, n, k, experts, _) in enumerate(KINDS):
    z = lambda *s, dtype=TYPES[dtype]: torch.zeros(*s, dtype=dtype, device="cuda")
    lead = (experts,) if experts else ()
    more = dict(offsets=torch.tensor(split(m, experts), dtype=torch.int32, device="cuda")) if experts else {}
    codes = z(*lead, n, (k + 31) // 32 * 16, dtype=torch.uint8)[..., :(k + 1) // 2]
    print("case", i, file=sys.stderr, flush=True)
    rx.rx_gemm_fp4(z(m, k), codes, z(*lead, n, (k + 63) // 64, dtype=torch.float32), z(m, n), 64, **more)
torch.cuda.synchronize()
"""


@pytest.mark.gpu
def test_sizes_select_every_kernel():
    """The names that the library reports of its launches, in a process that asks for them."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are for 256 CUs")
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, env=dict(os.environ, RX_DEBUG="1"), stdout=subprocess.PIPE,
                       stderr=subprocess.PIPE, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l for l in r.stderr.splitlines() if l.startswith("case ") or "k_gemm_fp4" in l]
    assert lines[::2] == [f"case {i}" for i in range(len(KINDS))]
    got = [l.split("k_gemm_fp4_")[1].split(" grid")[0] for l in lines[1::2]]
    assert got == [k[5] for k in KINDS]
    assert {(k[0], k[5]) for k in KINDS} >= {("fp32", n) for n in ("few", "stream 16x32", "stream 16x64", "stream 32x128", "parts")}
