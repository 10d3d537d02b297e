"""Plain float64 forms of the router, the products with 4-bit weights and the
layer norm (CPU torch), with error bounds counted from the roundings that the
float32 evaluation makes (as in block_ref.py: EPS32 is the most that one rounding
adds, relative to the value; a result's own rounding adds eps / 2 of its type).

expf and logf are within 2 units in the last place, 4 EPS32. x - max and x - lse
round once, which exp turns into a relative error of |difference| EPS32."""
import numpy as np
import torch

from block_ref import EPS32, cast_bound

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---- router --------------------------------------------------------------------

def route(logits, mask, topk, renormalize):
    """ids, and value and bound of weights and lse, of counts, and of the losses."""
    x = logits.double()
    t, e = x.shape
    live = ~torch.isinf(x).all(1) if e else torch.zeros(t, dtype=torch.bool)
    if mask is not None:
        live &= mask.bool()
    x = torch.where(live[:, None], x, torch.zeros_like(x))
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True)[1][:, :topk]
    top = x.gather(1, order)
    kept = live[:, None] & (top > -torch.inf)
    high = x.max(1, keepdim=True).values
    p = torch.softmax(x, 1)
    far = torch.where(p > 0, high - x, torch.zeros_like(x))
    # exp's argument and exp, additions within a lane (16) and between lanes (6),
    # division or multiplication with an inverse (3)
    mean = (p * far).sum(1, keepdim=True)
    rel = EPS32 * (far + mean + 40)
    chosen = torch.where(kept, p.gather(1, order), torch.zeros_like(top))
    share = torch.where(live, chosen.sum(1), torch.ones(t, dtype=torch.float64))[:, None] if renormalize else 1.0
    weights = chosen / share
    # the chosen ones' sum is one of up to 64 terms with the same kinds of error
    w_bound = weights * (rel.gather(1, order) + (EPS32 * (mean + far.gather(1, order).max(1, keepdim=True).values + 80) if renormalize else 0))
    w_bound = w_bound + 2.0 ** -148
    lse = torch.logsumexp(x, 1)
    lse_bound = EPS32 * (lse.abs() + (mean[:, 0] + 40) + 5 * (lse - high[:, 0]).abs())
    counts = torch.zeros(e + 1, dtype=torch.long)
    counts[:e] = torch.bincount(order[kept], minlength=e)
    counts[e] = live.sum()
    n = max(1, int(counts[e]))
    rate = counts[:e].double() / (n * topk)
    per = (p * live[:, None]).sum(0) / n
    balance = e * (rate * per).sum()
    # a sum over the tokens adds at most tokens / 64 + 64 numbers one after the other, one over the experts 64
    steps = t / 64 + 64 + 64 + 16
    b_bound = e * (rate * ((p * live[:, None]) * (rel + EPS32 * steps)).sum(0) / n).sum()
    z = (torch.where(live, lse.square(), torch.zeros_like(lse))).sum() / n
    z_bound = (torch.where(live, 2 * lse.abs() * lse_bound + lse.square() * EPS32 * steps, torch.zeros_like(lse))).sum() / n
    return dict(ids=torch.where(kept, order, -1).int(), weights=(weights, w_bound), lse=(torch.where(live, lse, -torch.inf), lse_bound),
                counts=counts.int(), losses=(torch.stack([balance, z]), torch.stack([b_bound, z_bound])), live=live, p=p,
                lse_value=lse, lse_err=lse_bound)


def route_backward(logits, f, d_weights, d_losses, renormalize, counts=None):
    """value and bound of d_logits from route()'s dict; counts may be others' too."""
    x = logits.double()
    t, e = x.shape
    ids, live, p = f["ids"].long(), f["live"], f["p"]
    topk = ids.shape[1]
    counts = f["counts"] if counts is None else counts
    n = max(1, int(counts[e]))
    kept = ids >= 0
    zero = torch.zeros_like(p)
    g = torch.where(kept, d_weights.double(), 0.0) if d_weights is not None else torch.zeros(t, topk, dtype=torch.float64)
    load = (d_losses[0].double() * e / n) * counts[:e].double() / (n * topk) if d_losses is not None else torch.zeros(e, dtype=torch.float64)
    zc = 2 * d_losses[1].double() / n if d_losses is not None else torch.zeros((), dtype=torch.float64)
    safe = ids.clamp(min=0)
    spread = lambda v: zero.scatter_add(1, safe, torch.where(kept, v, 0.0))
    if renormalize:
        pc = torch.where(kept, p.gather(1, safe), 0.0)
        share = pc.sum(1, keepdim=True)
        share = torch.where(share > 0, share, 1.0)
        mean = (pc * g).sum(1, keepdim=True) / share
        mean_abs = (pc * g.abs()).sum(1, keepdim=True) / share
        extra, extra_abs = spread((g - mean) / share), spread((g.abs() + mean_abs) / share)
        base, base_abs = load + zero, load.abs() + zero
    else:
        extra = extra_abs = zero
        base, base_abs = load + spread(g), load.abs() + spread(g.abs())
    lse = torch.where(live, f["lse_value"], 0.0)[:, None]
    d = p * (base - (p * base).sum(1, keepdim=True) + zc * lse + extra)
    size = p * (base_abs + (p * base_abs).sum(1, keepdim=True) + (zc * lse).abs() + extra_abs)
    # P twice or three times (exp(x - lse) with lse as it was stored), sums over a token, some twenty products
    far = torch.where(p > 0, (x - lse).abs(), 0.0).max(1, keepdim=True).values
    n_round = 3 * (far + 8) + 2 * 30 + 20
    bound = size * (EPS32 * n_round + 3 * f["lse_err"][:, None]) + 2.0 ** -140
    d = torch.where(live[:, None], d, 0.0)
    return d, cast_bound(d, torch.where(live[:, None], bound, 0.0), logits.dtype)


# ---- 4-bit weights -----------------------------------------------------------------

def quant_fp4(x, group):
    """codes (uint8, one an element), their values and the scales; the quotients and the product round to float32."""
    rows, k = x.shape
    groups = -(-k // group)
    padded = torch.zeros(rows, groups * group, dtype=torch.float64)
    padded[:, :k] = x.double()
    v = padded.view(rows, groups, group)
    top = v.abs().amax(2)
    s, r = (top / 6).float(), (6 / top).float()
    one = (top == 0) | (s == 0) | torch.isinf(r)
    s[one], r[one] = 1.0, 1.0
    y = (v * r.double()[:, :, None]).float().double().view(rows, -1)[:, :k]
    # the nearest level, ties to the even code: the borders at even codes belong to them
    code = torch.zeros(y.shape, dtype=torch.uint8)
    for c in range(1, 8):
        border = (LEVELS[c - 1] + LEVELS[c]) / 2
        code += (y.abs() >= border if c % 2 == 0 else y.abs() > border).to(torch.uint8)
    code += 8 * torch.signbit(y).to(torch.uint8)
    return code, s


def pack4(code):
    rows, k = code.shape
    full = torch.zeros(rows, (k + 1) // 2 * 2, dtype=torch.uint8)
    full[:, :k] = code
    return full[:, 0::2] | full[:, 1::2] << 4


def values4(code):
    return torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64)[code.long()]


def gemm_fp4(a, code, scales, group):
    """value and bound of a times the weights. Products are exact; a matrix instruction adds 32 products to a sum, in an
    order of its own (up to 32 roundings, each of up to a whole unit), up to four of them a group; then a rounding a
    group along k, and up to 16 sums of the parts of k."""
    k = a.shape[1]
    w = values4(code) * scales.double().repeat_interleave(group, 1)[:, :k]
    v = a.double() @ w.t()
    size = a.double().abs() @ w.abs().t()
    n = 2 * (4 * 32) + k / 32 + 16 + 8
    return v, cast_bound(v, n * EPS32 * size + 2.0 ** -126, a.dtype)


# ---- dropout and layer norm -----------------------------------------------------------

def philox(counter, key):
    """Philox of four words and ten rounds: rows of four words (numpy) under a key of two."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def kept(rows, hidden, drop, rng):
    """Which elements dropout keeps (rows x hidden), from seed and offset as a tensor of two int64."""
    seed, offset = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    per = -(-hidden // 8)
    i = np.arange(rows * per, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    full = lambda v: np.full(rows * per, v, dtype=np.uint64)
    words = philox(np.stack([i & low, i >> np.uint64(32), full(offset & 0xFFFFFFFF), full(offset >> 32)], 1),
                   (seed & 0xFFFFFFFF, seed >> 32))
    half = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(rows, per * 8)[:, :hidden]
    return torch.from_numpy(half.astype(np.int64)) >= threshold(drop)


def threshold(drop):
    return int(np.rint(np.float64(np.float32(drop)) * 65536))


def block_end(srcs, bias, residual, drop, rng):
    """value and bound of h before its rounding."""
    y = torch.stack([s.double() for s in srcs])
    v, m = y.sum(0), y.abs().sum(0)
    if bias is not None:
        v, m = v + bias.double(), m + bias.double().abs()
    if drop:
        p = threshold(drop) / 65536
        keep = kept(*v.shape, drop, rng).double() / (1 - p)
        # a dropped element is exactly 0, whatever it was
        v, m = (torch.where(keep > 0, t * keep, 0.0) for t in (v, m))
    if residual is not None:
        v, m = v + residual.double(), m + residual.double().abs()
    return v, (len(srcs) + 4) * EPS32 * m


def layer_norm(h, w, b, eps):
    """value and bound of z, mean and rstd from h as it is stored."""
    x = h.double()
    rows, n = x.shape
    adds = n / 64 + 24
    mean = x.mean(1, keepdim=True)
    mean_err = EPS32 * (adds + 2) * x.abs().mean(1, keepdim=True)
    c = x - mean
    c_err = EPS32 * c.abs() + mean_err
    var = (c * c).mean(1, keepdim=True)
    # of c's errors the common one adds its square (the c add up to 0), the roundings their share
    var_err = var * EPS32 * (adds + 6) + mean_err ** 2 + 2 * mean_err * EPS32 * c.abs().mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    rel = 0.5 * var_err / (var + eps) + 4 * EPS32
    one = torch.ones(n, dtype=torch.float64)
    wd, bd = one if w is None else w.double(), 0 * one if b is None else b.double()
    z = c * rstd * wd + bd
    # rel to first order: its square and c_err's product with it on top
    z_err = wd.abs() * rstd * (c_err * (1 + 2 * rel) + c.abs() * (rel + rel * rel)) + EPS32 * 3 * ((c * rstd * wd).abs() + bd.abs())
    return dict(z=(z, cast_bound(z, z_err, h.dtype)), mean=(mean[:, 0], mean_err[:, 0] + 0.0), rstd=(rstd[:, 0], (rstd * (rel + rel * rel))[:, 0]))


def layer_norm_backward(h, w, mean, rstd, d_h, d_z, drop, rng):
    """values, and bounds before the results' own rounding, from mean and rstd as they were stored."""
    shape = next(t for t in (h, d_h, d_z) if t is not None).shape
    rows, n = shape
    zero = torch.zeros(shape, dtype=torch.float64)
    dh = zero if d_h is None else d_h.double()
    if d_z is None:
        x = a = dz = zero
        q = torch.zeros(rows, 1, dtype=torch.float64)
    else:
        q = rstd.double()[:, None]
        x, dz = (h.double() - mean.double()[:, None]) * q, d_z.double()
        a = dz * (1.0 if w is None else w.double())
    mean_of = lambda t: t.mean(1, keepdim=True)
    full = dh + q * (a - mean_of(a) - x * mean_of(a * x))
    size = dh.abs() + q * (a.abs() + mean_of(a.abs()) + x.abs() * mean_of((a * x).abs()))
    n_row = n / 64 + 24 + 20
    err = n_row * EPS32 * size
    src, src_err, src_size = full, err, size
    if drop:
        keep = kept(rows, n, drop, rng).double() / (1 - threshold(drop) / 65536)
        src, src_err, src_size = full * keep, err * keep + 2 * EPS32 * (full * keep).abs(), size * keep
    n_sum = rows + 32
    return dict(d_residual=(full, err), d_src=(src, src_err), d_bias=(src.sum(0), src_err.sum(0) + n_sum * EPS32 * src_size.sum(0)),
                d_w=((dz * x).sum(0), (n_sum + 6) * EPS32 * (dz * x).abs().sum(0)), d_b=(dz.sum(0), n_sum * EPS32 * dz.abs().sum(0)))
