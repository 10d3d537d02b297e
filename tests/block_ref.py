"""Plain float64 forms of the operators around a block's allreduce (CPU torch),
with error bounds counted from the roundings that the float32 evaluation makes.

A bound is n * EPS32 * M: M is the operator's formula with every term taken
absolute, n the number of float32 roundings on the longest path from an input
to the result (a sum over a row of H elements goes through at most H / 64 + 24
additions in any lane-and-tree order a wave of 64 can take). Norms divide by a
root of a sum of squares, which amplifies the relative error of cancelled sums
by at most kappa = sum(M^2) / sum(value^2) of the row. A result's own rounding
adds eps / 2 of its type."""
import torch

EPS32 = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}   # float32 results: counted in n


def cast_bound(value, err, dtype):
    return err + HALF[dtype] * (value.abs() + err)


def plan(ids, first, experts):
    flat = ids.reshape(-1).tolist()
    local = [i - first if first <= i < first + experts else -1 for i in flat]
    order = [i for e in range(experts) for i, l in enumerate(local) if l == e]
    offsets = [0]
    for e in range(experts):
        offsets.append(offsets[-1] + local.count(e))
    slots = [-1] * len(flat)
    for p, i in enumerate(order):
        slots[i] = p
    order += [-1] * (len(flat) - len(order))
    i32 = torch.int32
    return torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32), \
        torch.tensor(slots, dtype=i32).reshape(ids.shape)


def gather(x, order, topk):
    rows = torch.zeros(order.numel(), x.shape[1], dtype=x.dtype)
    kept = order >= 0
    rows[kept] = x[order[kept].long() // topk]
    return rows


def quant_i8(x):
    """codes (int8) and scales (float32); the two quotients and the product round to float32."""
    x = x.double()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64)
    s, r = (top / 127).float(), (127 / top).float()
    one = (top == 0) | (s == 0) | torch.isinf(r)
    s[one], r[one] = 1.0, 1.0
    codes = torch.round((x * r.double()[:, None]).float())
    return codes.to(torch.int8), s


def gemm_i8(a, sa, b, sb, dtype):
    """value and bound: the sum's conversion and two products round to float32."""
    total = a.double() @ b.double().t()
    v = total * sa.double()[:, None] * sb.double()
    return v, cast_bound(v, 3.01 * EPS32 * v.abs() + 2.0 ** -149, dtype)


def combine(rows, slots, weights, nrows=None):
    nrows = rows.shape[0] if nrows is None else nrows
    t, k = slots.shape
    out = torch.zeros(t, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for i in range(t):
        for j in range(k):
            s = int(slots[i, j])
            if 0 <= s < nrows:
                w = 1.0 if weights is None else float(weights[i, j])
                out[i] += w * rows[s].double()
                mag[i] += (w * rows[s].double()).abs()
    return out, cast_bound(out, (k + 1) * 1.01 * EPS32 * mag, rows.dtype)


def combine_backward(d_out, rows, slots, weights, nrows):
    t, k = slots.shape
    h = d_out.shape[1]
    d_rows = torch.zeros(nrows, h, dtype=torch.float64)
    d_w = torch.zeros(t, k, dtype=torch.float64)
    m_w = torch.zeros(t, k, dtype=torch.float64)
    for i in range(t):
        for j in range(k):
            s = int(slots[i, j])
            if 0 <= s < nrows:
                w = 1.0 if weights is None else float(weights[i, j])
                d_rows[s] = w * d_out[i].double()
                if rows is not None:
                    prod = d_out[i].double() * rows[s].double()
                    d_w[i, j], m_w[i, j] = prod.sum(), prod.abs().sum()
    return d_rows, cast_bound(d_rows, 1.01 * EPS32 * d_rows.abs(), d_out.dtype), \
        d_w, (h / 64 + 25) * 1.01 * EPS32 * m_w


def norm(srcs, residual, gate, gate_rows, w_post, w_pre, rs, eps):
    """Every intermediate in float64, with the magnitudes of the absolute formula."""
    d = lambda t: None if t is None else t.double()
    x = torch.stack([s.double() for s in srcs])
    y, ym = x.sum(0), x.abs().sum(0)
    rows, h = y.shape
    idx = torch.arange(rows) // gate_rows
    g = d(gate)[idx] if gate is not None else torch.ones_like(y)
    res = d(residual) if residual is not None else torch.zeros_like(y)
    p = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if w_post is not None else torch.ones(rows, 1, dtype=torch.float64)
    wp = d(w_post) if w_post is not None else torch.ones(h, dtype=torch.float64)
    u, um = y * p * wp, ym * p * wp.abs()
    hh, hm = rs * res + g * u, (rs * res).abs() + g.abs() * um
    q = 1 / torch.sqrt((hh * hh).mean(1, keepdim=True) + eps)
    wz = d(w_pre) if w_pre is not None else torch.ones(h, dtype=torch.float64)
    tiny = 1e-300
    kappa = torch.ones(rows, 1, dtype=torch.float64)
    if w_post is not None:
        kappa = kappa * ((ym * ym).mean(1, keepdim=True) + eps) / ((y * y).mean(1, keepdim=True) + eps + tiny)
    kappa = kappa * ((hm * hm).mean(1, keepdim=True) + eps) / ((hh * hh).mean(1, keepdim=True) + eps + tiny)
    z, zm = hh * q * wz, hm * q * wz.abs()
    return dict(y=y, ym=ym, p=p, u=u, um=um, g=g, h=hh, hm=hm, q=q, wp=wp, wz=wz, z=z, zm=zm, kappa=kappa, idx=idx,
                # fold, two sums over the row with root and quotient, products
                n=len(srcs) + 2 * (h / 64 + 24) + 24)


def norm_backward(f, d_h, d_z, rs, post, groups):
    """Gradients from norm()'s dict, and their bounds before the results' own rounding."""
    y, p, q, h, g, wp, wz = (f[k] for k in ("y", "p", "q", "h", "g", "wp", "wz"))
    n_el = y.shape[1]
    zero = torch.zeros_like(y)
    dh = d_h.double() if d_h is not None else zero
    dz = d_z.double() if d_z is not None else zero
    a = dz * wz
    full = dh + q * (a - h * q * q * (a * h).mean(1, keepdim=True))
    fm = dh.abs() + q * (a.abs() + f["hm"] * q * q * (a.abs() * f["hm"]).mean(1, keepdim=True))
    du, dum = full * g, fm * g.abs()
    if post:
        b, bm = du * wp, dum * wp.abs()
        dy = p * (b - y * p * p * (b * y).mean(1, keepdim=True))
        dym = p * (bm + f["ym"] * p * p * (bm * f["ym"]).mean(1, keepdim=True))
    else:
        dy, dym = du, dum
    k = f["kappa"]
    # a second row sum after the forward's two, and the products around them
    n = (f["n"] + h.shape[1] / 64 + 24 + 24) * EPS32
    rows = y.shape[0]
    nr = n + (rows + 32) * EPS32   # a sum over the rows on top
    out = dict(d_src=(dy, n * k * dym), d_residual=(rs * full, n * k * abs(rs) * fm),
               d_w_pre=((dz * h * q).sum(0), nr * (k * dz.abs() * f["hm"] * q).sum(0)),
               d_w_post=((du * y * p).sum(0), nr * (k * dum * f["ym"] * p).sum(0)))
    if groups:
        dg, dgm = torch.zeros(groups, n_el, dtype=torch.float64), torch.zeros(groups, n_el, dtype=torch.float64)
        dg.index_add_(0, f["idx"], full * f["u"])
        dgm.index_add_(0, f["idx"], k * fm * f["um"])
        out["d_gate"] = (dg, nr * dgm)
    return out
