"""Plain 64-bit forms of the operators beside kda_fwd, token by token and slot by slot, with
bounds on how far 32-bit arithmetic may be from them (what the GPU tests compare against).

The bounds. u = 2^-24 is half a step of fp32. In the recurrence every token multiplies the
state by exp(g) and adds x. An exp computed as 2^(g log2 e) is off by at most 2u of its value
plus 2u|g| from rounding the exponent, a product or a fused multiply-add by u of the absolute
sum, and taking the tokens in groups whose affine maps are composed adds at most four more
roundings a token: STEP(g) = (8 + 2|g|) u of the sum of absolute terms, carried along by the
recurrence itself. Rounding the result to its type adds half a step of it.

An exp(g) below the smallest normal fp32 number (g < -87.3) may come out as zero: it is then
off by less than TINY = 2^-126, so the state before, of absolute sum s, adds less than TINY s
(and to dg, which multiplies by h_{t-1}, TINY s |h_{t-1}|: s and h can each be above one, so
the smallest normal number alone does not cover it).
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def spans(cu, B, T):
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return [(int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1)]


def glr(x, g, sp, h0=None, dy=None, d_final=None):
    """x, g, dy [tokens, D] (any float type); h0, d_final [N, D]. Returns dicts of values and of
    bounds: y, final, before (the state that enters each token) and, with dy, dx, dg, d_initial."""
    f = torch.float64
    x, g = x.to(f), g.to(f)
    a, step = g.exp(), (8 + 2 * torch.where(torch.isinf(g), 0.0, g.abs())) * U
    D, n = x.shape[1], len(sp)
    z = torch.zeros(n, D, dtype=f)
    h0 = z if h0 is None else h0.to(f)
    v = {"y": torch.zeros_like(x), "final": h0.clone(), "before": torch.zeros_like(x)}
    e = {k: torch.zeros_like(t) for k, t in v.items()}
    for i, (b, t1) in enumerate(sp):
        h, s, err = h0[i].clone(), h0[i].abs(), torch.zeros(D, dtype=f)
        for t in range(b, t1):
            v["before"][t], e["before"][t] = h, err
            h = a[t] * h + x[t]
            lost = TINY * s
            s = a[t] * s + x[t].abs()
            err = a[t] * err + step[t] * s + lost
            v["y"][t], e["y"][t] = h, err
        v["final"][i], e["final"][i] = h, err
    if dy is None:
        return v, e
    dy = dy.to(f)
    d_final = z if d_final is None else d_final.to(f)
    for k in ("dx", "dg"):
        v[k], e[k] = torch.zeros_like(x), torch.zeros_like(x)
    v["d_initial"], e["d_initial"] = d_final.clone(), torch.zeros(n, D, dtype=f)
    for i, (b, t1) in enumerate(sp):
        E, s, err = d_final[i].clone(), d_final[i].abs(), torch.zeros(D, dtype=f)
        for t in range(t1 - 1, b - 1, -1):
            G, s = dy[t] + E, s + dy[t].abs()
            err = err + U * s
            v["dx"][t], e["dx"][t] = G, err
            lost = TINY * s
            E, s = a[t] * G, a[t] * s
            err = a[t] * err + step[t] * s + lost
            v["dg"][t] = E * v["before"][t]
            e["dg"][t] = err * v["before"][t].abs() + (E.abs() + err) * e["before"][t] + 2 * U * v["dg"][t].abs()
        v["d_initial"][i], e["d_initial"][i] = E, err
    return v, e


def assert_near(name, got, want, bound):
    """got within bound of want, and half a step of its type for the rounding at the end. The
    smallest normal number of the type is what flushed or gradual underflow may cost."""
    got64 = got.detach().cpu().to(torch.float64).reshape(want.shape)
    tol = bound + half_step(got.dtype) * (want.abs() + bound) + torch.finfo(got.dtype).tiny
    bad = ~((got64 - want).abs() <= tol)
    if bool(bad.any()):
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got "
                             f"{got64.reshape(-1)[i].item()!r}, want {want.reshape(-1)[i].item()!r}, "
                             f"tolerance {tol.reshape(-1)[i].item():.3e}")


def depth(n):
    """Roundings that a sum of n terms takes at most: a lane adds up to n / 64 of them one after
    the other (one lane each for short rows), and at most 64 partial sums follow."""
    return min(n, 64 + n / 64 + 64)


def layernorm(x, w, b, eps):
    """Values and bounds of y, mean, rstd. A mean of D terms is off by depth(D) u of their mean
    absolute value; centred values by that and u of x; the variance is a sum of squares of
    those; each of the products after it adds u."""
    f = torch.float64
    x = x.to(f)
    D = x.shape[1]
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = (c.square().mean(1, keepdim=True) + eps) ** -0.5
    w, b = (torch.ones(D, dtype=f) if w is None else w.to(f)), (torch.zeros(D, dtype=f) if b is None else b.to(f))
    y = c * rstd * w + b
    k = (depth(D) + 4) * U
    dm = k * x.abs().mean(1, keepdim=True)
    dc = dm + U * x.abs()
    # var: 2 c dc, its sum's roundings, dm^2; rstd: half the relative error of var + eps
    dvar = 2 * (c.abs() * dc).mean(1, keepdim=True) + dc.square().mean(1, keepdim=True) + k * c.square().mean(1, keepdim=True)
    drel = 0.5 * dvar * rstd.square() + 4 * U
    # beyond the first order: (1 + d)^(-1/2) for d up to 1/2
    drel = torch.where(dvar * rstd.square() < 0.5, drel * 1.5, torch.full_like(drel, float("inf")))
    dy = w.abs() * rstd * (dc * (1 + drel) + c.abs() * drel) + 4 * U * ((c * rstd * w).abs() + b.abs())
    return ({"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}, {"y": dy, "mean": dm[:, 0], "rstd": (rstd * drel)[:, 0]})


def layernorm_bwd(dy, x, w, mean, rstd):
    """Values and bounds of dx, dw, db from given fp32 mean and rstd."""
    f = torch.float64
    dy, x, r, m = dy.to(f), x.to(f), rstd.to(f)[:, None], mean.to(f)[:, None]
    M, D = x.shape
    w = torch.ones(D, dtype=f) if w is None else w.to(f)
    xh = (x - m) * r
    dxh = 3 * U * r * (x.abs() + m.abs())
    a = dy * w
    c1, c2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    k = (depth(D) + 4) * U
    d1 = k * a.abs().mean(1, keepdim=True)
    d2 = k * (a * xh).abs().mean(1, keepdim=True) + (a.abs() * dxh).mean(1, keepdim=True)
    dx = r * (a - c1 - xh * c2)
    ddx = r * (d1 + xh.abs() * d2 + dxh * (c2.abs() + d2) + 6 * U * (a.abs() + c1.abs() + (xh * c2).abs()))
    # the sums over rows go through at most 1 + M / 64 additions in a lane or a part of the
    # workspace, 1024 parts in a row, and what rows share inside a workgroup
    km = min(M, 64 + M / 64 + 1024) + 4
    v = {"dx": dx, "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    e = {"dx": ddx, "dw": (dy.abs() * dxh).sum(0) + km * U * (dy * xh).abs().sum(0), "db": km * U * dy.abs().sum(0)}
    return v, e


def fork(used, src):
    """(dst, used after): lists of ints."""
    used, before, dst = list(used), list(used), []
    for s in src:
        free = [i for i, u in enumerate(used) if not u]
        if not free or not (s == -1 or (0 <= s < len(used) and before[s])):
            dst.append(-1)
            continue
        used[free[0]] = 1
        dst.append(free[0])
    return dst, used


def compact(used):
    """(moves [(from, to)], remap)."""
    n = sum(1 for u in used if u)
    to = [i for i in range(n) if not used[i]]
    of = [i for i in range(n, len(used)) if used[i]]
    assert len(to) == len(of)
    remap = [i if u else -1 for i, u in enumerate(used)]
    for a, b in zip(of, to):
        remap[a] = b
    return list(zip(of, to)), remap
