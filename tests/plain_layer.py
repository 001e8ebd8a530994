"""Plain 64-bit forms of the norm, the convolution and the scan, with bounds on how far 32-bit
arithmetic may be from them (what the GPU tests compare against).

The bounds are a running error analysis: an `R` is a value with a bound on how far what 32 bits
compute may be from it. u = 2^-24 is half a step of fp32. Every operation passes on the bounds of
what it takes and adds its own rounding: u of a sum, a product or a fused multiply-add, 2u + 2u|x|
of an exponential computed as 2^(x log2 e) (one step of the instruction, and the rounding of the
exponent), 2u of a reciprocal. A sum of n terms in whatever order is off by at most n u of the sum
of their sizes. Results of what fp32 flushes or underflows are off by at most TINY, its smallest
normal number.
"""
import torch

from plain_ops import TINY, U, assert_near, half_step, spans  # noqa: F401

f64 = torch.float64


class R:
    def __init__(self, v, e=None):
        self.v = v.to(f64) if isinstance(v, torch.Tensor) else torch.tensor(float(v), dtype=f64)
        self.e = torch.zeros_like(self.v) if e is None else e

    def _round(self, k=1):
        return R(self.v, self.e + k * U * (self.v.abs() + self.e) + TINY)

    def __add__(self, o):
        o = o if isinstance(o, R) else R(o)
        return R(self.v + o.v, self.e + o.e)._round()

    def __neg__(self):
        return R(-self.v, self.e)

    def __sub__(self, o):
        return self + (-(o if isinstance(o, R) else R(o)))

    def __mul__(self, o):
        o = o if isinstance(o, R) else R(o)
        return R(self.v * o.v, self.v.abs() * o.e + o.v.abs() * self.e + self.e * o.e)._round()

    __radd__, __rmul__ = __add__, __mul__

    def __getitem__(self, i):
        return R(self.v[i], self.e[i])

    def view(self, *s):
        return R(self.v.reshape(*s), self.e.reshape(*s))

    def exp(self):
        v = self.v.exp()
        return R(v, v * (torch.expm1(self.e) + (2 + 2 * self.v.abs()) * U * torch.exp(self.e)) + TINY)

    def sum(self, dim, keepdim=False):
        n = self.v.shape[dim]
        v = self.v.sum(dim, keepdim=keepdim)
        return R(v, self.e.sum(dim, keepdim=keepdim) + (n + 1) * U * (self.v.abs() + self.e).sum(dim, keepdim=keepdim) + TINY)


def sigmoid(x):
    """1 / (1 + exp(-|x|)), or that times the exponential: the quotient's size is at most 1."""
    v = torch.sigmoid(x.v)
    e = (4 + 2 * x.v.abs()) * U + 4 * U
    # d sigmoid = s (1 - s) dx; relative roundings of the exponential, the sum and the reciprocal
    return R(v, v * torch.sigmoid(-x.v) * x.e * 1.5 + v * e + 32 * TINY)


def silu(x):
    """x sigmoid(x); the exponential of a number beyond 88 is infinite, its quotient 0 (32 TINY
    covers x exp(x) there)."""
    s = sigmoid(x)
    v = x.v * s.v
    return R(v, 1.1 * x.e + x.v.abs() * s.v * (8 + 2 * x.v.abs()) * U + 32 * TINY)._round()


def dsilu(x):
    """s (1 + x (1 - s)); its derivative is at most 1/2."""
    s = torch.sigmoid(x.v)
    inner = 1 + x.v * (1 - s)
    size = s * (1 + x.v.abs() * (1 - s))
    # s, 1 - s and the product: 1 - s is off by the absolute error of s, s (8 + 2|x|) u, times |x|
    err = size * (10 + 2 * x.v.abs()) * U + s * x.v.abs() * s * (8 + 2 * x.v.abs()) * U
    return R(s * inner, 0.5 * x.e + err + 64 * TINY * (1 + x.v.abs()))


def softplus(x):
    """max(x, 0) + log(1 + exp(-|x|)): the logarithm's series and quotient add at most 10 u of it."""
    e = torch.exp(-x.v.abs())
    lg = torch.log1p(e)
    v = x.v.clamp(min=0) + lg
    return R(v, torch.sigmoid(x.v) * x.e * 1.5 + lg * (14 + 2 * x.v.abs()) * U + TINY)._round(2)


def cat(rs):
    return R(torch.cat([r.v for r in rs]), torch.cat([r.e for r in rs]))


def stack(rs, dim=0):
    return R(torch.stack([r.v for r in rs], dim), torch.stack([r.e for r in rs], dim))


# ---- root-mean-square norm ----------------------------------------------------------------


def rmsnorm(x, residual, w, eps):
    """R of the sum s, rstd and y."""
    s = R(x) if residual is None else R(x) + R(residual)
    D = s.v.shape[1]
    w = R(torch.ones(D) if w is None else w)
    q = (s * s).sum(1, keepdim=True) * (1.0 / D)
    q = R(q.v, q.e + U * q.v) + eps
    rel = torch.where(q.v > 0, q.e / q.v, 1.0)
    # (1 + d)^(-1/2) for |d| up to 1/2: at most d; the root and the quotient 2u each
    r = R(q.v ** -0.5, q.v ** -0.5 * (torch.where(rel < 0.5, rel, float("inf")) + 4 * U))
    return s, R(r.v[:, 0], r.e[:, 0]), s * r * w


def rmsnorm_bwd(dy, x, w, rstd, d_residual):
    """R of dx and dw from given fp32 rstd."""
    dy, x, r = R(dy), R(x), R(rstd)
    r = R(r.v[:, None])
    a = dy if w is None else dy * R(w)
    xh = x * r
    D = x.v.shape[1]
    mean = (a * xh).sum(1, keepdim=True) * (1.0 / D)
    dx = r * (a - xh * R(mean.v, mean.e + 2 * U * mean.v.abs()))
    if d_residual is not None:
        dx = dx + R(d_residual)
    return dx, (dy * xh).sum(0)


# ---- short causal convolution ---------------------------------------------------------------


def conv(x, w, b, sp, h0=None, use_silu=True, dy=None, d_final=None):
    """x, dy [tokens, D]; w [D, W]; h0, d_final [N, W - 1, D] or None. Dicts of R: y, final and, with
    dy, dx, dw, db, d_initial. Tokens outside sp are NaN in y and dx."""
    D, W = w.shape
    n, w = len(sp), R(w)
    b = R(torch.zeros(D)) if b is None else R(b)
    h0 = torch.zeros(n, W - 1, D) if h0 is None else h0
    nan = torch.full((x.shape[0], D), float("nan"), dtype=f64)
    y, dx = R(nan.clone()), R(nan.clone())
    fin, dini, dws, dbs = [], [], [], []
    for i, (lo, hi) in enumerate(sp):
        v = cat([R(h0[i]), R(x[lo:hi])])
        L = hi - lo
        fin.append(v[L:])
        if dy is not None:
            dv = R(torch.zeros(L + W - 1, D))
            if d_final is not None:
                dv = R(torch.cat([dv.v[:L], d_final[i].to(f64)]))
        if L > 0:
            u = b
            for j in range(W):
                u = u + w[:, j] * v[j:j + L]
            o = silu(u) if use_silu else u
            y.v[lo:hi], y.e[lo:hi] = o.v, o.e
        if dy is None:
            continue
        if L > 0:
            du = R(dy[lo:hi])
            if use_silu:
                du = du * dsilu(u)
            for j in range(W):
                t = dv[j:j + L] + w[:, j] * du
                dv.v[j:j + L], dv.e[j:j + L] = t.v, t.e
            dws.append(stack([du * v[j:j + L] for j in range(W)], 2))
            dbs.append(du)
            dx.v[lo:hi], dx.e[lo:hi] = dv.v[W - 1:], dv.e[W - 1:]
        dini.append(dv[:W - 1])
    out = {"y": y, "final": stack(fin)}
    if dy is not None:
        zero = R(torch.zeros(1, D, W)), R(torch.zeros(1, D))
        out.update(dx=dx, dw=cat([zero[0]] + dws).sum(0), db=cat([zero[1]] + dbs).sum(0), d_initial=stack(dini))
    return out


# ---- selective state space scan ---------------------------------------------------------------


def ssm(x, dt, A, B, C, sp, skip=None, z=None, bias=None, use_softplus=True, h0=None, dy=None, d_final=None):
    """x, dt, z, dy [tokens, D]; A [D, E]; B, C [tokens, G, E]; h0, d_final [N, D, E] or None. Dicts
    of R as the operator's outputs. Tokens outside sp are NaN.

    Chunks of the tokens pass states by exp(A sum s): rounding a sum of up to T terms is off by T u
    of it, so the exponent of a token's decay carries T u |s A| besides its own roundings, and
    composing adds at most 4 u a token."""
    T, D = x.shape
    E, G, n = A.shape[1], B.shape[1], len(sp)
    x, A, rB, rC = R(x), R(A), R(B), R(C)
    pre = R(dt) if bias is None else R(dt) + R(bias)
    s = softplus(pre) if use_softplus else pre
    ex = R(s.v[:, :, None]) * A
    arg = R(ex.v, ex.e + s.e[:, :, None] * A.v.abs() + (T + 4) * U * ex.v.abs())
    a = arg.exp()
    a = R(a.v, a.e + 4 * U * a.v)
    wide = lambda m: R(m.v.repeat_interleave(D // G, 1), m.e.repeat_interleave(D // G, 1))  # noqa: E731
    Bw, Cw = wide(rB), wide(rC)
    sx = s * x
    u = R(sx.v[:, :, None], sx.e[:, :, None]) * Bw
    zero = torch.zeros(n, D, E, dtype=f64)
    h0 = zero if h0 is None else h0.to(f64)
    new = lambda *sh: R(torch.full(sh, float("nan"), dtype=f64))  # noqa: E731
    h, before = new(T, D, E), new(T, D, E)
    fin = R(h0.clone())

    def put(r, i, v):
        r.v[i], r.e[i] = v.v, v.e
    for i, (lo, hi) in enumerate(sp):
        c = R(h0[i])
        for t in range(lo, hi):
            put(before, t, c)
            c = a[t] * c + u[t]
            put(h, t, c)
        put(fin, i, c)
    y0 = (Cw * h).sum(2)
    if skip is not None:
        y0 = y0 + R(skip) * x
    out = {"y": y0 if z is None else y0 * silu(R(z)), "final": fin}
    if dy is None:
        return out
    dy = R(dy)
    g = dy if z is None else dy * silu(R(z))
    if z is not None:
        out["dz"] = dy * y0 * dsilu(R(z))
    S, Sa = new(T, D, E), new(T, D, E)
    dini = R(zero.clone() if d_final is None else d_final.to(f64).clone())
    gC = R(g.v[:, :, None], g.e[:, :, None]) * Cw
    for i, (lo, hi) in enumerate(sp):
        c = dini[i]
        for t in range(hi - 1, lo - 1, -1):
            c = c + gC[t]
            put(S, t, c)
            c = a[t] * c
            put(Sa, t, c)
        put(dini, i, c)
    used = torch.zeros(T, dtype=torch.bool)
    for lo, hi in sp:
        used[lo:hi] = True
    q = Sa * before
    SB = (S * Bw).sum(2)
    groups = lambda r: R(r.v.view(T, G, D // G, E), r.e.view(T, G, D // G, E))  # noqa: E731
    out["dC"] = groups(R(g.v[:, :, None], g.e[:, :, None]) * h).sum(2)
    out["dB"] = groups(R(sx.v[:, :, None], sx.e[:, :, None]) * S).sum(2)
    pad = lambda r: R(torch.cat([r.v[used], torch.zeros_like(r.v[:1])]), torch.cat([r.e[used], torch.zeros_like(r.v[:1])]))  # noqa: E731
    out["dA"] = pad(R(s.v[:, :, None], s.e[:, :, None]) * q).sum(0)
    dx = s * SB
    ds = (q * A).sum(2) + x * SB
    if skip is not None:
        dx = dx + R(skip) * g
        out["dskip"] = pad(g * x).sum(0)
    ddt = ds * sigmoid(pre) if use_softplus else ds
    out.update(dx=dx, ddt=ddt, d_initial=dini)
    if bias is not None:
        out["dbias"] = pad(ddt).sum(0)
    return out


def near(name, got, r, rows=None):
    """got within r's bound, the rounding to its type besides; rows: only these of the first dimension."""
    want, bound = r.v.reshape(got.shape), r.e.reshape(got.shape)
    if rows is not None:
        got, want, bound = got[rows], want[rows], bound[rows]
    assert_near(name, got, want, bound)


# ---- beams ---------------------------------------------------------------------------------------


def beam(logits, scores, k, finished=None, eos=0):
    """tokens, parents [N][k] and scores (64 bits) by sorting all continuations."""
    N, W, V = logits.shape
    tokens, parents, best = [], [], []
    for n in range(N):
        found = []
        for b in range(W):
            s = float(scores[n, b])
            x = logits[n, b].to(f64)
            if finished is not None and int(finished[n, b]):
                cand = {eos: s}
            else:
                top = x.max()   # (x - (top + log sum) would lose the sum beside a top of 1e38)
                lse = torch.log(torch.exp(x - top).sum())
                v = ((x - top) - lse) + s
                ok = torch.isfinite(v) & bool(torch.isfinite(lse))
                cand = {int(i): float(v[i]) for i in ok.nonzero()[:, 0]} if V <= 64 or k >= V else None
                if cand is None:
                    v = torch.where(ok, v, -float("inf"))
                    best_of = torch.sort(v, descending=True, stable=True)
                    cand = {int(i): float(q) for q, i in zip(best_of.values[:k], best_of.indices[:k]) if torch.isfinite(q)}
            found += [(-q, b, v) for v, q in cand.items() if q == q and abs(q) != float("inf")]
        found = sorted(found)[:k]
        found += [(float("inf"), -1, -1)] * (k - len(found))
        tokens.append([f[2] for f in found])
        parents.append([f[1] for f in found])
        best.append([-f[0] for f in found])
    return tokens, parents, best


def reorder(pool, slots, parents):
    """New slots [N][W] and the pool after it (pool [L, S, ...], lists of lists)."""
    S, after, out = pool.shape[1], pool.clone(), []
    for sl, pa in zip(slots, parents):
        W, seen, new, rest = len(sl), set(), [None] * len(sl), []
        for j, p in enumerate(pa):
            if 0 <= p < W and p not in seen:
                seen.add(p)
                new[j] = sl[p]
            else:
                rest.append(j)
        free = [b for b in range(W) if b not in seen]
        for j, b in zip(rest, free):
            new[j] = sl[b]
            if 0 <= pa[j] < W and 0 <= sl[b] < S and 0 <= sl[pa[j]] < S:
                after[:, sl[b]] = pool[:, sl[pa[j]]]
        out.append(new)
    return out, after
