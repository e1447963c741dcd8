"""Float64 definitions of the routed layer's gradients, and error bounds counted from
the roundings that a float32 computation makes (u = 2^-24 each).  Plain torch on the
inputs' device; nothing of the library is used."""
import math

import torch

U = 2.0 ** -24


def half_step(ref, dtype):
    """What one rounding of ref to dtype may cost: half an epsilon of the value, or half
    a step below the smallest normal number."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) * (1 + 2.0 ** -7) + f.tiny * f.eps / 2


def close(got, ref, slack, what=""):
    """|got - ref| <= slack + one rounding of (|ref| + slack) to got's type."""
    assert got.shape == ref.shape, what
    ref, slack = ref.double(), torch.as_tensor(slack, dtype=torch.float64, device=ref.device)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    err = (got.double() - ref).abs()
    room = slack + half_step(ref.abs() + slack, got.dtype)
    bad = (err > room) & ~nan & (got.double() != ref)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()} for {ref[i].item()}, {err[i].item()} over "
                             f"{room.expand_as(err)[i].item()}")


# ------------------------------------------------------------------ tokens and routes
def combine_backward(d_out, y, w, r2r, scale):
    """(d_y, d_w, their slacks); rows that no route names are NaN in d_y."""
    T, H = d_out.shape
    K = w.shape[1]
    M = T * K
    d, y, w = d_out.double(), y.double(), w.double().flatten()
    d_y = torch.full((M, H), math.nan, dtype=torch.float64, device=d.device)
    d_w = torch.zeros(M, dtype=torch.float64, device=d.device)
    s_w = torch.zeros_like(d_w)
    for r in range(M):
        row = int(r2r[r])
        if 0 <= row < M:
            d_y[row] = scale * w[r] * d[r // K]
            t = d[r // K] * y[row]
            d_w[r], s_w[r] = scale * t.sum(), scale * t.abs().sum()
    # scale * w and its product with d; a lane's chain of H / 32 terms, the tree, the scale
    return d_y, d_w.view(T, K), 2 * U * d_y.abs(), (H / 32 + 16) * U * s_w.view(T, K).abs()


def permute_backward(d_x, r2r, K):
    M, H = d_x.shape
    out = torch.zeros((M // K, H), dtype=torch.float64, device=d_x.device)
    mag = torch.zeros_like(out)
    for r in range(M):
        row = int(r2r[r])
        if 0 <= row < M:
            out[r // K] += d_x[row].double()
            mag[r // K] += d_x[row].double().abs()
    return out, K * U * mag


# ------------------------------------------------------------------ activation
def split(p, kind, inter):
    if kind in ("relu", "identity", "gelu1", "silu1"):
        return p, None
    if inter:
        return p[:, 0::2], p[:, 1::2]
    return p[:, :p.shape[1] // 2], p[:, p.shape[1] // 2:]


def join(g, u, inter):
    if u is None:
        return g
    return torch.stack((g, u), 2).flatten(1) if inter else torch.cat((g, u), 1)


def cdf(x):
    return 0.5 * torch.erfc(x * -(0.5 ** 0.5))


def pdf(x):
    return torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)


def act_forward(p, kind, inter=False, limit=0.0, alpha=1.0, beta=0.0):
    """act(p) in float64 (kinds: silu, gelu, swiglu gated; silu1, gelu1, relu, identity)."""
    g, u = split(p.double(), kind, inter)
    if kind == "identity":
        return g.clone()
    if kind == "relu":
        return torch.where(g > 0, g, g * 0)
    if kind in ("gelu", "gelu1"):
        return g * cdf(g) * (1 if u is None else u)
    if kind == "swiglu":
        if limit > 0:
            g, u = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
        return g * torch.sigmoid(alpha * g) * (u + beta)
    return g * torch.sigmoid(g) * (1 if u is None else u)


def act_backward(p, d, kind, inter=False, limit=0.0, alpha=1.0, beta=0.0, fast=False):
    """(act, slack of act, d_p, slack of d_p).  The slack counts the sigmoid's relative
    error: 8 u exact, (8 + 1.2 |x|) 2^-23 with the fast exponential (its stated bound)
    and quotient; products and sums 8 u of their terms' magnitudes.

    These are relative and hold for normal numbers only.  A factor (sigmoid, Phi, a product
    of two factors) below 2^-126 is a multiple of 2^-149, off by a few of these (erfc's four
    units in the last place, and one rounding a product: 2^-146).  The fast quotient gives
    zero for results below 2^-126, and the exact sigmoid 1 / (1 + exp(-x)) below 2^-128, where
    the exponential overflows: off by 2^-126 at most.  The other factors, at most
    (1 + |d|) (1 + |g|) (1 + |u|), multiply that."""
    p, d = p.double(), d.double()
    g, u = split(p, kind, inter)
    one = torch.ones_like(g)
    sigmoid = kind in ("silu", "silu1", "swiglu")
    low = 2.0 ** -125 if fast or sigmoid else 2.0 ** -146
    low = low * (1 + g.abs()) * (1 + (0 if u is None else u.abs()))
    low_d = low * (1 + d.abs())
    a = act_forward(p, kind, inter, limit, alpha, beta)
    if kind == "identity":
        return a, 0 * a, d, 0 * a
    if kind == "relu":
        return a, 0 * a, torch.where(g > 0, d, 0 * g), 0 * a
    if kind in ("gelu", "gelu1"):
        w = one if u is None else u
        c, f = cdf(g), pdf(g)
        # the exponent and erfc's argument are rounded: a relative 2 u g^2 of pdf, g pdf u of cdf
        dc = 8 * U * c + 4 * U * g.abs() * f
        df = f * (8 + 2 * g * g) * U
        # fast: exp(-x^2 / 2) to (2 + 1.2 x^2 / 2) 2^-23, its cofactor of the lower tail to 2^-19
        if fast:
            df = df + f * (2 + 0.6 * g * g) * 2 * U
            tail = torch.minimum(c, cdf(-g))
            dc = tail * (2.0 ** -19 + (2 + 0.6 * g * g) * 2 * U + (12 + g * g) * U) + U
            dc = torch.where(g < 0, dc - U, dc)
        s_a = (g * w).abs() * (dc + 4 * U * c) + low
        dg = d * w * (c + g * f)
        s_g = (d * w).abs() * (dc + g.abs() * df + 8 * U * (c + (g * f).abs())) + low_d
        du, s_u = d * g * c, (d * g).abs() * (dc + 4 * U * c) + low_d
        return (a, s_a, dg, s_g) if u is None else (a, s_a, join(dg, du, inter),
                                                    join(s_g, s_u, inter))
    gg, uu, al = g, one if u is None else u, 1.0
    pass_g = pass_u = torch.ones_like(g, dtype=torch.bool)
    if kind == "swiglu":
        al = alpha
        if limit > 0:
            pass_g, pass_u = ~(g > limit), ~(u.abs() > limit)
            gg, uu = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
        uu = uu + beta
    x = al * gg
    s = torch.sigmoid(x)
    rel = (8 + 1.2 * x.abs()) * 2 * U if fast else (8 + x.abs()) * U
    rel = rel + 8 * U
    dg = torch.where(pass_g, d * uu * s * (1 + x * (1 - s)), 0 * g)
    s_g = (d * uu).abs() * s * (1 + x.abs()) * rel * 2 + U * d.abs() * s * (1 + x.abs()) + low_d
    du = torch.where(pass_u, d * gg * s, 0 * g)
    s_u = torch.where(pass_u, du.abs() * rel + low_d, 0 * g)
    # u + beta is rounded once: u |u + beta| is in rel
    s_a = a.abs() * rel + low
    if u is None:
        return a, s_a, dg, s_g
    return a, s_a, join(dg, du, inter), join(torch.where(pass_g, s_g, 0 * g), s_u, inter)


# ------------------------------------------------------------------ grouped products
def bounds(seg_end, M):
    """[(lo, hi)] of every expert, clamped as the kernels clamp."""
    out, lo = [], 0
    ends = seg_end.tolist()
    for i, e in enumerate(ends):
        lo = 0 if i == 0 else max(0, min(ends[i - 1], M))
        out.append((lo, max(lo, min(e, M))))
    return out


def dgrad(d, w, seg_end):
    """(d_a, slack); rows outside every segment are NaN.  A sum of n exact products in
    float32, tensor cores cutting what they shift out: n 2^-23 of the magnitudes."""
    M, N = d.shape
    out = torch.full((M, w.shape[2]), math.nan, dtype=torch.float64, device=d.device)
    mag = torch.zeros_like(out)
    for e, (lo, hi) in enumerate(bounds(seg_end, M)):
        out[lo:hi] = d[lo:hi].double() @ w[e].double()
        mag[lo:hi] = d[lo:hi].double().abs() @ w[e].double().abs()
    return out, (N + 2) * 2 * U * mag


def wgrad(d, a, seg_end):
    """(d_w, slack, d_bias, slack)."""
    M, N = d.shape
    E = seg_end.numel()
    out = torch.zeros((E, N, a.shape[1]), dtype=torch.float64, device=d.device)
    mag, b = torch.zeros_like(out), torch.zeros((E, N), dtype=torch.float64, device=d.device)
    bmag = torch.zeros_like(b)
    for e, (lo, hi) in enumerate(bounds(seg_end, M)):
        x, y = d[lo:hi].double(), a[lo:hi].double()
        out[e], mag[e] = x.t() @ y, (hi - lo + 2) * 2 * U * (x.abs().t() @ y.abs())
        b[e], bmag[e] = x.sum(0), (hi - lo + 2) * U * x.abs().sum(0)
    return out, mag, b, bmag


# ------------------------------------------------------------------ router
def route_weights(z, ids, scoring, renorm, rsf):
    """topk_weights in float64; ids outside [0, E) weigh nothing."""
    if scoring == "softmax":
        s = torch.softmax(z, 1)
    elif scoring == "sigmoid":
        s = torch.sigmoid(z)
    else:
        s = torch.sqrt(torch.nn.functional.softplus(z, threshold=700.0))  # (smooth at zero)
    ok = (ids >= 0) & (ids < z.shape[1])
    s = torch.where(ok, s.gather(1, torch.where(ok, ids, 0).long()), 0.0)
    return rsf * (s / s.sum(1, keepdim=True) if renorm else s)


def route_backward(z, ids, g, scoring, renorm, rsf):
    """(d_logits, slack): every term c v l g carries the relative errors of two
    exponentials of arguments up to max |z - m|, a quotient and a few products."""
    z = z.double().detach().requires_grad_()
    w = route_weights(z, ids, scoring, renorm, rsf)
    d = torch.autograd.grad((w * g.double()).sum(), z)[0]
    with torch.no_grad():
        ok = (ids >= 0) & (ids < z.shape[1])
        gw = torch.where(ok, w * g.double().abs(), 0.0)
        mag = torch.zeros_like(z).scatter_add(1, torch.where(ok, ids, 0).long(), gw)
        # the sum's part: w_k times sum_j |g_j| w_j / rsf, on every expert for a plain softmax
        total = gw.sum(1, keepdim=True) / rsf
        if scoring == "softmax" and not renorm:
            mag = mag + rsf * torch.softmax(z, 1) * total
        elif renorm:
            mag = mag + torch.zeros_like(z).scatter_add(1, torch.where(ok, ids, 0).long(),
                                                        torch.where(ok, w, 0.0)) * total
        # float64 differentiation leaves its own rounding, 2^-53 of a few terms, where the
        # softmax's sum cancels and the gradient is zero
        noise = 2.0 ** -50 * rsf * total if scoring == "softmax" else 0.0
        span = 2 * z.abs().amax(1, keepdim=True).clamp(max=200)
        return d, (40 + 2 * ids.shape[1] + 4 * span) * U * mag + noise
