"""What the operators of a state space layer and of its serving are measured on.

  conv    the short causal convolution before a recurrence, per channel over the last 2 to 4
          tokens, with SiLU: forward ("fwd"), forward and backward ("train"), one token per
          sequence with the last inputs in slots of a cache ("step");
  ssm     the selective state space scan, E states per channel:
          h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t, y_t = (C_t . h_t + D x_t) SiLU(z_t):
          forward ("fwd"), forward and backward ("train"), one token per sequence ("step");
  rms     the root-mean-square norm of a residual stream: the layer's output added, the sum
          normed, rounded to the input's type or to 8 bits with a scale for each 128 elements
          or each row ("fwd"); backward with the weight's gradient ("bwd");
  beam    a step of beam search: the best continuations of every sequence's beams over the
          vocabulary, and the beams' states in a cache made to follow them ("step").

A case's sizes are the KDA workloads' own (8192 tokens, 64 heads of 128, 8 heads as one
GPU's share of them, 256 sequences in generation, 32 ragged sequences) or generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
MOST = 8192 * 8192             # elements of one of the largest token tensors
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "none": 0}
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
TOP = 448.0                    # the largest e4m3 value


def listed():
    return [
        # one token for each of a few sequences, an odd width: the latency of a call
        {"name": "conv step, 3 sequences", "op": "conv", "kind": "step", "N": 3, "D": 129, "W": 4, "dtype": "fp32", "state": "fp32"},
        # prefill of one long sequence, 64 heads of 128 channels
        {"name": "conv forward, 8192 tokens", "op": "conv", "kind": "fwd", "B": 1, "T": 8192, "N": 0, "D": 8192, "W": 4, "dtype": "bf16", "state": "none"},
        # a training step on 32 packed sequences of ragged lengths, one GPU's share of 8 heads
        {"name": "conv training, ragged", "op": "conv", "kind": "train", "B": 1, "T": 26810, "N": 32, "D": 1024, "W": 4, "dtype": "bf16", "state": "bf16"},
        # a generation step of 256 sequences, 64 heads of 128 channels with 16 states each
        {"name": "ssm step, 256 sequences", "op": "ssm", "kind": "step", "N": 256, "D": 8192, "E": 16, "G": 1, "dtype": "bf16", "state": "fp32"},
        # prefill of one long sequence, 64 heads of 128 channels
        {"name": "ssm forward, 8192 tokens", "op": "ssm", "kind": "fwd", "B": 1, "T": 8192, "N": 0, "D": 8192, "E": 16, "G": 1, "dtype": "bf16", "state": "none"},
        # a training step on 32 packed sequences of ragged lengths, one GPU's share of 8 heads
        {"name": "ssm training, ragged", "op": "ssm", "kind": "train", "B": 1, "T": 26810, "N": 32, "D": 1024, "E": 16, "G": 1, "dtype": "bf16", "state": "fp32"},
        # a training step on two rows of 4096 tokens, B and C shared by the channels of four groups
        {"name": "ssm training, 2 x 4096", "op": "ssm", "kind": "train", "B": 2, "T": 4096, "N": 0, "D": 4096, "E": 16, "G": 4, "dtype": "bf16", "state": "none"},
        # the norm of a few tokens in generation, its output in 8 bits for the product after it
        {"name": "rms forward, 5 rows", "op": "rms", "kind": "fwd", "M": 5, "D": 4096, "dtype": "bf16", "residual": True, "out": "row"},
        # the norm before a layer in prefill, its output in 8 bits with a scale for each 128
        {"name": "rms forward, 8 bits", "op": "rms", "kind": "fwd", "M": 8192, "D": 8192, "dtype": "bf16", "residual": True, "out": "block"},
        # its backward pass in training, with the gradient that comes along the residual stream
        {"name": "rms backward, wide", "op": "rms", "kind": "bwd", "M": 8192, "D": 8192, "dtype": "bf16", "residual": True, "out": "same"},
        # one sequence with 4 beams, an odd vocabulary, the states of one GPU's share of 8 heads
        {"name": "beam step, 1 x 4", "op": "beam", "kind": "step", "N": 1, "W": 4, "V": 32003, "k": 4, "dtype": "fp32", "L": 1, "slot": 8 * 128 * 128, "state": "bf16"},
        # 32 sequences with 8 beams each, a large vocabulary, the states of 8 heads in two layers
        {"name": "beam step, 32 x 8", "op": "beam", "kind": "step", "N": 32, "W": 8, "V": 131072, "k": 8, "dtype": "bf16", "L": 2, "slot": 8 * 128 * 128, "state": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, kind = rng.choice([("conv", "step"), ("conv", "fwd"), ("conv", "train"), ("ssm", "step"), ("ssm", "fwd"), ("ssm", "train"),
                           ("rms", "fwd"), ("rms", "bwd"), ("beam", "step"), ("beam", "step")])
    c = {"op": op, "kind": kind}
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "rms":
        c["D"] = _log(rng, 32, 16384)
        c["M"] = _log(rng, 1, max(1, MOST // 2 // c["D"]))
        c.update(dtype=dtype, residual=rng.random() < 0.7, out=rng.choice(["same", "block", "row"]) if kind == "fwd" else "same")
        return c
    if op == "beam":
        c.update(W=_log(rng, 1, 16), V=_log(rng, 500, 131072))
        c["N"] = _log(rng, 1, max(1, min(64, (1 << 25) // (c["W"] * c["V"]))))
        c["k"] = c["W"]
        c.update(dtype=dtype, L=rng.randint(1, 3), slot=_log(rng, 64, max(64, min(1 << 18, (1 << 27) // (c["N"] * c["W"])))), state=rng.choice(["fp32", "bf16"]))
        return c
    if op == "ssm":
        c["E"] = rng.choice([16, 16, 8, _log(rng, 1, 64)])
        c["G"] = rng.choice([1, 1, 2, 5])
        c["D"] = c["G"] * (8 * _log(rng, 2, 8192 // 8 // c["G"]) if rng.random() < 0.7 else _log(rng, 13, 8192 // c["G"]))
        most = min(32768, MOST * 16 // 4 // (c["D"] * c["E"]), MOST // 4 // c["D"])
    else:
        c["W"] = rng.randint(2, 4)
        c["D"] = 8 * _log(rng, 8, 1024) if rng.random() < 0.7 else _log(rng, 64, 8192)
        most = min(32768, MOST // 2 // c["D"])
    if kind == "step":
        c.update(N=_log(rng, 1, 256), dtype=dtype, state=rng.choice(["fp32", "bf16"]))
        return c
    T = _log(rng, 16, max(16, most))
    if rng.random() < 0.5:
        c.update(B=1, T=T, N=_log(rng, 1, min(64, T)))
    else:
        B = _log(rng, 1, 4)
        c.update(B=B, T=max(1, T // B), N=0)
    c.update(dtype=dtype, state=rng.choice(["none", "fp32", "bf16"]))
    return c


# ---- inputs -----------------------------------------------------------------


def _normal(gen, shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)


def _uniform(gen, shape, lo, hi):
    return torch.rand(shape, generator=gen, device=DEV) * (hi - lo) + lo


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _new(shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _bounds(case, rng):
    """Lengths of case["N"] packed sequences, log-uniform over a factor of 64, one in eight empty when they are many."""
    n, T = case["N"], case["T"]
    w = np.exp(rng.uniform(0, math.log(64), n))
    if n > 8:
        w[rng.permutation(n)[: n // 8]] = 0
    cu = np.concatenate([[0], np.round(np.cumsum(w) / w.sum() * T)]).astype(np.int64)
    cu[-1] = T
    return cu


def _rows_of(case, rng):
    """Number of sequences, their boundaries on the GPU and on the host (of rows too)."""
    if case["N"]:
        cu = _bounds(case, rng)
        return case["N"], torch.from_numpy(cu).to(DEV), cu.tolist()
    return case["B"], None, [b * case["T"] for b in range(case["B"] + 1)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 31))
    op, kind = case["op"], case["kind"]
    t, st = TYPES[case["dtype"]], TYPES.get(case.get("state"))
    s = {"case": case}
    if op == "rms":
        M, D = case["M"], case["D"]
        like = _uniform(gen, (D,), 0.5, 2.5)
        s.update(x=(_normal(gen, (M, D)) * like).to(t), w=_normal(gen, (D,), std=0.2, mean=1.0), rstd=_new(M))
        if kind == "bwd":   # x is the residual stream that the forward pass has left, rstd its norm's
            s["rstd"] = (1 / torch.sqrt(s["x"].double().square().mean(1) + EPS)).float()
            s.update(dy=_normal(gen, (M, D), t), dres=_normal(gen, (M, D), t) if case["residual"] else None,
                     dx=_new((M, D), t), dw=_new(D))
            return s
        if case["residual"]:
            s.update(res=(_normal(gen, (M, D), std=2.0) * like).to(t), res_out=_new((M, D), t))
        if case["out"] == "same":
            s["y"] = _new((M, D), t)
        else:
            s.update(y=_new((M, D), E4M3), scales=_new((M, -(-D // 128) if case["out"] == "block" else 1)))
        return s
    if op == "beam":
        N, W, V, k = case["N"], case["W"], case["V"], case["k"]
        slots = rng.permutation(N * W + 3)[: N * W].reshape(N, W)
        s.update(logits=_normal(gen, (N, W, V), t, std=3.0), scores=-_uniform(gen, (N, W), 5.0, 8.0), slots=_ints(slots),
                 tokens=_new((N, k), torch.int32), parents=_new((N, k), torch.int32), new_scores=_new((N, k)),
                 new_slots=_new((N, W), torch.int32), pool=_normal(gen, (case["L"], N * W + 3, case["slot"]), st, std=0.02))
        return s
    D = case["D"]
    if op == "conv":
        W = case["W"]
        s.update(w=_uniform(gen, (D, W), -1.0, 1.0) / math.sqrt(W), b=_normal(gen, (D,), std=0.1))
    else:
        E, G = case["E"], case["G"]
        lo = _uniform(gen, (D,), math.log(1e-3), math.log(0.1)).exp()   # dt at the start of training
        s.update(A=-(torch.arange(1, E + 1, device=DEV) * _uniform(gen, (D, E), 0.8, 1.25)), skip=_normal(gen, (D,), std=0.1, mean=1.0),
                 bias=lo + torch.log(-torch.expm1(-lo)))
    if kind == "step":
        N = case["N"]
        slots = rng.permutation(2 * N)   # the states before the step stay in their slots
        s.update(x=_normal(gen, (N, D), t), y=_new((N, D), t), src=_ints(slots[:N]), dst=_ints(slots[N:]))
        if op == "conv":
            s["pool"] = _normal(gen, (2 * N, case["W"] - 1, D), st)
        else:
            s.update(dt=_normal(gen, (N, D), t, std=0.7), z=_normal(gen, (N, D), t), Bm=_normal(gen, (N, G, E), t),
                     Cm=_normal(gen, (N, G, E), t), pool=_normal(gen, (2 * N, D, E), st, std=0.3))
        return s
    B, T = case["B"], case["T"]
    n, cu, host = _rows_of(case, rng)
    s.update(x=_normal(gen, (B, T, D), t), y=_new((B, T, D), t), cu=cu, cu_host=host)
    train = kind == "train"
    if train:
        s.update(dy=_normal(gen, (B, T, D), t), dx=_new((B, T, D), t))
    if op == "conv":
        shape = (n, case["W"] - 1, D)
        if train:
            s.update(dw=_new((D, case["W"])), db=_new(D))
    else:
        shape = (n, D, E)
        s.update(dt=_normal(gen, (B, T, D), t, std=0.7), z=_normal(gen, (B, T, D), t), Bm=_normal(gen, (B, T, G, E), t),
                 Cm=_normal(gen, (B, T, G, E), t), carry=None)
        if train:
            s.update(ddt=_new((B, T, D), t), dz=_new((B, T, D), t), dB=_new((B, T, G, E), t), dC=_new((B, T, G, E), t),
                     dA=_new((D, E)), dskip=_new(D), dbias=_new(D), carry=_new((-(-B * T // 64), D, E)))
    s.update(h0=None if st is None else _normal(gen, shape, st, std=0.3), hT=_new(shape, st or torch.float32))
    if train:
        s.update(dhT=_normal(gen, shape), dh0=_new(shape))
    return s


# ---- the plain forms: 32 bits, rounded once at the end -------------------------


def _ends(s):
    """Sequences that hold tokens, and the packed places of their first and last ones."""
    cu = torch.tensor(s["cu_host"], device=DEV) if s["cu"] is None else s["cu"]
    some = cu[1:] > cu[:-1]
    return some, cu[:-1][some], cu[1:][some] - 1


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _padded(s, W):
    """Packed inputs with each sequence's W - 1 inputs of before it in front of them, and where each token and each end lies there."""
    D = s["x"].shape[-1]
    cu = torch.tensor(s["cu_host"], device=DEV) if s["cu"] is None else s["cu"]
    n, total = cu.numel() - 1, s["x"].numel() // D
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), cu[1:] - cu[:-1], output_size=total)
    at = torch.arange(total, device=DEV) + (W - 1) * (seq + 1)
    front = (cu[:-1] + (W - 1) * torch.arange(n, device=DEV))[:, None] + torch.arange(W - 1, device=DEV)   # [n, W - 1]
    v = torch.zeros(total + n * (W - 1), D, device=DEV)
    v[at] = s["x"].reshape(-1, D).float()
    if s["h0"] is not None:
        v[front] = s["h0"].float()
    return v, at, front, front + (cu[1:] - cu[:-1])[:, None]


def _conv_plain(s):
    c, x = s["case"], s["x"]
    W, D = c["W"], x.shape[-1]
    v, at, front, back = _padded(s, W)
    u = s["b"] + sum(v[at - (W - 1 - j)] * s["w"][:, j] for j in range(W))
    sg = _sigmoid(u)
    out = {"y": (u * sg).to(x.dtype).view(x.shape), "final": v[back].to(s["hT"].dtype)}
    if c["kind"] == "fwd":
        return out
    du = s["dy"].reshape(-1, D).float() * (sg * (1 + u * (1 - sg)))
    out["dw"] = torch.stack([(du * v[at - (W - 1 - j)]).sum(0) for j in range(W)], 1)
    out["db"] = du.sum(0)
    del u, sg
    wide = torch.zeros_like(v)   # the outputs' gradients at the padded places
    wide[at] = du
    dv = torch.zeros_like(v)
    for j in range(W):           # an input serves the outputs at its place and the W - 1 after it
        o = W - 1 - j
        dv[: v.shape[0] - o] += wide[o:] * s["w"][:, j]
    dv.index_put_((back,), s["dhT"], accumulate=True)
    out.update(dx=dv[at].to(x.dtype).view(x.shape), d_initial=dv[front])
    return out


def _conv_step_plain(s):
    W = s["case"]["W"]
    v = torch.cat([s["pool"][s["src"].long()].float(), s["x"].float()[:, None]], 1)
    u = s["b"] + (v * s["w"].t()[None]).sum(1)
    s["pool"][s["dst"].long()] = v[:, 1:].to(s["pool"].dtype)
    return {"y": (u * _sigmoid(u)).to(s["x"].dtype), "pool": s["pool"]}


def _softplus(u):
    return torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs()))


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 0, by doubling: after the step of length s each entry holds 2s tokens."""
    s = 1
    while s < a.shape[0]:
        u = torch.cat([u[:s], a[s:] * u[:-s] + u[s:]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return u


def _wide(m, D):
    """B or C of [..., G, E] for every channel: [tokens, D, E], of stride 0 over the channels of a group."""
    G, E = m.shape[-2:]
    return m.reshape(-1, G, 1, E).float().expand(-1, G, D // G, E)


def _ssm_plain(s):
    c, x = s["case"], s["x"].reshape(-1, s["x"].shape[-1]).float()
    D, E, G, t = c["D"], c["E"], c["G"], s["x"].dtype
    shape = s["x"].shape
    some, first, last = _ends(s)
    n = some.numel()
    h0 = torch.zeros(n, D, E, device=DEV) if s["h0"] is None else s["h0"].float()
    pre = s["dt"].reshape(-1, D).float() + s["bias"]
    dt = _softplus(pre)
    a = torch.exp(dt[:, :, None] * s["A"])
    u = ((dt * x).view(-1, G, D // G, 1) * _wide(s["Bm"], D)).view(-1, D, E)
    u[first] += a[first] * h0[some]
    cut = a.clone()   # decays that do not reach over the start of a sequence
    cut[first] = 0
    h = _scan(cut, u)
    del u
    hT = h0.clone()
    hT[some] = h[last]
    y0 = (h.view(-1, G, D // G, E) * _wide(s["Cm"], D)).sum(-1).view(-1, D) + s["skip"] * x
    z = s["z"].reshape(-1, D).float()
    sg = _sigmoid(z)
    out = {"y": (y0 * z * sg).to(t).view(shape), "final": hT.to(s["hT"].dtype)}
    if c["kind"] == "fwd":
        return out
    # with g = dy SiLU(z): G_t = C_t g_t + a_{t+1} G_{t+1}
    dy = s["dy"].reshape(-1, D).float()
    g = dy * z * sg
    out["dz"] = (dy * y0 * (sg * (1 + z * (1 - sg)))).to(t).view(shape)
    del y0, sg, dy
    out["dskip"] = (g * x).sum(0)
    out["dC"] = (g.view(-1, G, D // G, 1) * h.view(-1, G, D // G, E)).sum(2).to(t).view(s["Cm"].shape)
    v = (g.view(-1, G, D // G, 1) * _wide(s["Cm"], D)).view(-1, D, E)
    v[last] += s["dhT"][some]
    after = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    del cut
    S = _scan(after.flip(0), v.flip(0)).flip(0)
    del after, v
    out["dB"] = ((dt * x).view(-1, G, D // G, 1) * S.view(-1, G, D // G, E)).sum(2).to(t).view(s["Bm"].shape)
    SB = (S.view(-1, G, D // G, E) * _wide(s["Bm"], D)).sum(-1).view(-1, D)
    out["dx"] = (s["skip"] * g + dt * SB).to(t).view(shape)
    S = S * a
    del a
    dh0 = s["dhT"].clone()
    dh0[some] = S[first]
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = h0[some]
    S = S * before
    del before, h
    out["dA"] = (S * dt[:, :, None]).sum(0)
    dpre = ((S * s["A"]).sum(-1) + x * SB) * _sigmoid(pre)
    out.update(ddt=dpre.to(t).view(shape), dbias=dpre.sum(0), d_initial=dh0)
    return out


def _ssm_step_plain(s):
    c = s["case"]
    D, E, G = c["D"], c["E"], c["G"]
    x, z = s["x"].float(), s["z"].float()
    dt = _softplus(s["dt"].float() + s["bias"])
    h = torch.exp(dt[:, :, None] * s["A"]) * s["pool"][s["src"].long()].float()
    h = h + ((dt * x).view(-1, G, D // G, 1) * _wide(s["Bm"], D)).reshape(-1, D, E)
    y = (h.view(-1, G, D // G, E) * _wide(s["Cm"], D)).sum(-1).view(-1, D) + s["skip"] * x
    s["pool"][s["dst"].long()] = h.to(s["pool"].dtype)
    return {"y": (y * z * _sigmoid(z)).to(s["x"].dtype), "pool": s["pool"]}


def _rms_plain(s):
    c, x, w = s["case"], s["x"].float(), s["w"]
    if c["kind"] == "bwd":
        r, a = s["rstd"][:, None], s["dy"].float() * w
        dx = r * (a - x * r.square() * (a * x).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(s["x"].dtype), "dw": (s["dy"].float() * x * r).sum(0)}
    out = {}
    if c["residual"]:
        x = x + s["res"].float()
        out["res_out"] = x.to(s["x"].dtype)
    rstd = 1 / torch.sqrt(x.square().mean(1) + EPS)
    y = x * rstd[:, None] * w
    out["rstd"] = rstd
    if c["out"] == "same":
        out["y"] = y.to(s["x"].dtype)
        return out
    M, D = y.shape
    size = 128 if c["out"] == "block" else D
    k = -(-D // size)
    y = torch.nn.functional.pad(y, (0, k * size - D)).view(M, k, size)
    scale = y.abs().amax(2) / TOP
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    out["scales"] = scale
    out["y"] = (y / scale[..., None]).clamp(-TOP, TOP).to(E4M3).view(M, k * size)[:, :D].contiguous()
    return out


def _follow_plain(s, parents):
    """Where the beams' states are: the first child of a beam stays in its slot, the others get copies in the slots of beams without children."""
    slots, p = s["slots"], parents.long()
    of = p[:, :, None] == torch.arange(slots.shape[1], device=DEV)                  # [N, child, beam]
    first = torch.gather(of.cumsum(1), 2, p[:, :, None])[..., 0] == 1
    free = torch.sort(of.any(1).to(torch.int8), dim=1, stable=True).indices          # beams without children first, ascending
    rank = ((~first).cumsum(1) - 1).clamp(min=0)
    old = torch.gather(slots, 1, p)
    new = torch.where(first, old, torch.gather(slots, 1, torch.gather(free, 1, rank)))
    s["pool"][:, new[~first].long()] = s["pool"][:, old[~first].long()]
    return new


def _beam_plain(s):
    k, (N, W, V) = s["case"]["k"], s["logits"].shape
    v = s["logits"].double()     # 64 bits: continuations of different beams lie close together
    top = v.amax(-1, keepdim=True)
    v = (v - top) - torch.log(torch.exp(v - top).sum(-1, keepdim=True)) + s["scores"].double()[..., None]
    v, at = torch.sort(v.view(N, W * V), dim=1, descending=True, stable=True)
    v, at = v[:, :k], at[:, :k]
    parents = (at // V).to(torch.int32)
    return {"scores": v.float(), "tokens": (at % V).to(torch.int32), "parents": parents, "slots": _follow_plain(s, parents), "pool": s["pool"]}


# ---- one pass -------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    op, kind = c["op"], c["kind"]
    if not own:
        if op == "conv":
            return _conv_step_plain(s) if kind == "step" else _conv_plain(s)
        if op == "ssm":
            return _ssm_step_plain(s) if kind == "step" else _ssm_plain(s)
        return _rms_plain(s) if op == "rms" else _beam_plain(s)
    import gated_delta_rule_87_amd as kda
    if op == "conv" and kind == "step":
        kda.conv_step(s["x"], s["w"], s["b"], s["y"], s["pool"], s["src"], s["dst"])
        return {"y": s["y"], "pool": s["pool"]}
    if op == "conv":
        kda.conv_fwd(s["x"], s["w"], s["b"], s["y"], initial_state=s["h0"], final_state=s["hT"], cu_seqlens=s["cu"])
        out = {"y": s["y"], "final": s["hT"]}
        if kind == "train":
            kda.conv_bwd(s["x"], s["w"], s["b"], s["dy"], s["dx"], d_weight=s["dw"], d_bias=s["db"], initial_state=s["h0"],
                         d_final=s["dhT"], d_initial=s["dh0"], cu_seqlens=s["cu"])
            out.update(dx=s["dx"], dw=s["dw"], db=s["db"], d_initial=s["dh0"])
        return out
    if op == "ssm" and kind == "step":
        kda.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["y"], s["pool"], s["src"], s["dst"], D=s["skip"], z=s["z"],
                     dt_bias=s["bias"])
        return {"y": s["y"], "pool": s["pool"]}
    if op == "ssm":
        kda.ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["y"], D=s["skip"], z=s["z"], dt_bias=s["bias"],
                    initial_state=s["h0"], final_state=s["hT"], cu_seqlens=s["cu"], carry=s["carry"])
        out = {"y": s["y"], "final": s["hT"]}
        if kind == "train":
            kda.ssm_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], s["carry"], s["dx"], s["ddt"], s["dA"], s["dB"], s["dC"],
                        D=s["skip"], d_D=s["dskip"], z=s["z"], d_z=s["dz"], dt_bias=s["bias"], d_dt_bias=s["dbias"],
                        initial_state=s["h0"], d_final=s["dhT"], d_initial=s["dh0"], cu_seqlens=s["cu"])
            out.update(dx=s["dx"], ddt=s["ddt"], dA=s["dA"], dB=s["dB"], dC=s["dC"], dskip=s["dskip"], dz=s["dz"], dbias=s["dbias"],
                       d_initial=s["dh0"])
        return out
    if op == "rms" and kind == "bwd":
        kda.rmsnorm_bwd(s["dy"], s["x"], s["w"], s["rstd"], s["dx"], d_weight=s["dw"], d_residual=s["dres"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "rms":
        kda.rmsnorm_fwd(s["x"], s["w"], EPS, s["y"], residual=s.get("res"), residual_out=s.get("res_out"), scales=s.get("scales"),
                        rstd=s["rstd"])
        out = {"y": s["y"], "rstd": s["rstd"]}
        if c["residual"]:
            out["res_out"] = s["res_out"]
        if c["out"] != "same":
            out["scales"] = s["scales"]
        return out
    kda.beam_select(s["logits"], s["scores"], s["tokens"], s["parents"], s["new_scores"])
    kda.cache_reorder(s["pool"], s["slots"], s["parents"], s["new_slots"])
    return {"scores": s["new_scores"], "tokens": s["tokens"], "parents": s["parents"], "slots": s["new_slots"], "pool": s["pool"]}


def work(case):
    op, kind = case["op"], case["kind"]
    t, st = SIZE[case["dtype"]], SIZE[case.get("state", "none")]
    if op == "rms":
        n, M, D = case["M"] * case["D"], case["M"], case["D"]
        if kind == "bwd":
            return {"bytes": n * t * (4 if case["residual"] else 3) + 4 * M + 8 * D, "flops": n * 11}
        y = n * t if case["out"] == "same" else n + 4 * M * (1 if case["out"] == "row" else -(-D // 128))
        return {"bytes": n * t * (3 if case["residual"] else 1) + y + 4 * M + 4 * D, "flops": n * (5 if case["out"] == "same" else 8)}
    if op == "beam":
        N, W, V, k = case["N"], case["W"], case["V"], case["k"]
        moved = N * max(0, W - 1) / 2   # about half of the beams come from another one's state
        return {"bytes": N * W * V * t + N * W * 16 + N * k * 12 + 2 * moved * case["L"] * case["slot"] * st, "flops": 4 * N * W * V}
    D = case["D"]
    if kind == "step":
        N = case["N"]
        if op == "conv":
            return {"bytes": N * D * (2 * t + 2 * (case["W"] - 1) * st) + 4 * D * (case["W"] + 1) + 8 * N, "flops": N * D * (2 * case["W"] + 5)}
        E = case["E"]
        return {"bytes": N * D * (4 * t + 2 * E * st) + 2 * N * case["G"] * E * t + 4 * D * (E + 2) + 8 * N, "flops": N * D * (8 * E + 12)}
    n, rows, train = case["B"] * case["T"] * D, case["N"] or case["B"], kind == "train"
    if op == "conv":
        W = case["W"]
        state, params = rows * (W - 1) * D, 4 * D * (W + 1)
        return {"bytes": n * t * (2 + 3 * train) + state * (st + (st or 4) + 8 * train) + params * (1 + 2 * train),
                "flops": n * (2 * W + 5 + train * (6 * W + 9))}
    E = case["E"]
    state, shared, params = rows * D * E, 2 * case["B"] * case["T"] * case["G"] * E * t, 4 * D * (E + 2)
    return {"bytes": n * t * (4 + 7 * train) + shared * (1 + 2 * train) + state * (st + (st or 4) + 8 * train) + params * (1 + 2 * train),
            "flops": n * ((7 + 16 * train) * E + 12 + 20 * train)}


# ---- the definition in 64 bits ----------------------------------------------------


def exact(case, seed):
    op, kind = case["op"], case["kind"]
    s = prepare(case, seed)
    f = torch.float64
    if op == "beam":
        x = s["logits"].to(f)
        x = x - torch.logsumexp(x, -1, keepdim=True) + s["scores"].to(f)[..., None]
        return {"scores": x.flatten(1).topk(case["k"], dim=1).values, "tokens": None, "parents": None, "slots": None, "pool": None}
    if op == "rms":
        x, w, D = s["x"].to(f), s["w"].to(f), case["D"]
        if kind == "bwd":
            xh = x * s["rstd"].to(f)[:, None]
            p = s["dy"].to(f) * w
            dx = (p - xh * ((p * xh).sum(1, keepdim=True) / D)) * s["rstd"].to(f)[:, None]
            return {"dx": dx if s["dres"] is None else dx + s["dres"].to(f), "dw": (s["dy"].to(f) * xh).sum(0)}
        out = {}
        if case["residual"]:
            out["res_out"] = x = x + s["res"].to(f)
        out["rstd"] = ((x * x).sum(1) / D + EPS) ** -0.5
        out["y"] = x * out["rstd"][:, None] * w
        if case["out"] != "same":   # the values before they are rounded to 8 bits, in units of their scale
            cols = range(0, D, 128 if case["out"] == "block" else D)
            step = cols.step
            out["scales"] = torch.stack([out["y"][:, i:i + step].abs().max(1).values for i in cols], 1) / TOP
            out["y"] = torch.cat([out["y"][:, i:i + step] / out["scales"][:, j:j + 1] for j, i in enumerate(cols)], 1)
        return out
    silu = lambda v: v * torch.sigmoid(v)  # noqa: E731
    dsilu = lambda v: torch.sigmoid(v) * (1 + v * torch.sigmoid(-v))  # noqa: E731
    D, x = case["D"], s["x"].to(f)
    if op == "conv":
        W, w, b = case["W"], s["w"].to(f), s["b"].to(f)
        if kind == "step":
            pool, y = s["pool"].to(f), torch.empty_like(x)
            for i, (p, q) in enumerate(zip(s["src"].tolist(), s["dst"].tolist())):
                v = torch.cat([s["pool"][p].to(f), x[i][None]])
                y[i] = silu(b + torch.einsum("jd,dj->d", v, w))
                pool[q] = v[1:]
            return {"y": y, "pool": pool}
        cu, x = s["cu_host"], x.reshape(-1, D)
        n = len(cu) - 1
        h0 = torch.zeros(n, W - 1, D, dtype=f, device=DEV) if s["h0"] is None else s["h0"].to(f)
        y, hT, dx, dh0 = torch.empty_like(x), h0.clone(), torch.empty_like(x), torch.empty_like(h0)
        dw, db = torch.zeros(D, W, dtype=f, device=DEV), torch.zeros(D, dtype=f, device=DEV)
        for i in range(n):
            lo, hi = cu[i], cu[i + 1]
            v = torch.cat([h0[i], x[lo:hi]])
            L = hi - lo
            u = b.expand(L, D).clone()
            for j in range(W):
                u += w[:, j] * v[j:j + L]
            y[lo:hi], hT[i] = silu(u), v[L:]
            if kind == "train":
                du, dv = s["dy"].reshape(-1, D)[lo:hi].to(f) * dsilu(u), torch.zeros_like(v)
                dv[L:] = s["dhT"][i].to(f)
                for j in range(W):
                    dv[j:j + L] += du * w[:, j]
                    dw[:, j] += (du * v[j:j + L]).sum(0)
                db += du.sum(0)
                dx[lo:hi], dh0[i] = dv[W - 1:], dv[:W - 1]
        out = {"y": y.view(s["x"].shape), "final": hT}
        if kind == "train":
            out.update(dx=dx.view(s["x"].shape), dw=dw, db=db, d_initial=dh0)
        return out
    E, G, A = case["E"], case["G"], s["A"].to(f)
    pre = s["dt"].to(f).reshape(-1, D) + s["bias"].to(f)
    dt = torch.where(pre > 0, pre, 0.0) + torch.log1p(torch.exp(-pre.abs()))
    x, z, skip = x.reshape(-1, D), s["z"].to(f).reshape(-1, D), s["skip"].to(f)
    Bm, Cm = (s[k].to(f).reshape(-1, G, E).repeat_interleave(D // G, 1) if kind == "step" else s[k].to(f).reshape(-1, G, E) for k in ("Bm", "Cm"))
    if kind == "step":
        pool, y = s["pool"].to(f), torch.empty_like(x)
        for i, (p, q) in enumerate(zip(s["src"].tolist(), s["dst"].tolist())):
            pool[q] = torch.exp(dt[i][:, None] * A) * s["pool"][p].to(f) + (dt[i] * x[i])[:, None] * Bm[i]
            y[i] = ((pool[q] * Cm[i]).sum(1) + skip * x[i]) * silu(z[i])
        return {"y": y, "pool": pool}
    # token by token, each sequence from its first token and back from its last
    cu, dx_in = s["cu_host"], dt * x
    n, total, train = len(cu) - 1, x.shape[0], kind == "train"
    hT = torch.zeros(n, D, E, dtype=f, device=DEV) if s["h0"] is None else s["h0"].to(f)
    h0 = hT.clone()
    y = torch.empty_like(x)
    kept = torch.empty(total if train else 1, D, E, dtype=f, device=DEV)
    by = lambda v: v.view(G, D // G, E)  # noqa: E731
    for i in range(n):
        h = h0[i].clone()
        for k in range(cu[i], cu[i + 1]):
            h = torch.addcmul(by(torch.exp(dt[k][:, None] * A) * h), dx_in[k].view(G, -1, 1), Bm[k][:, None]).view(D, E)
            y[k] = torch.bmm(by(h), Cm[k][:, :, None]).view(D)
            if train:
                kept[k] = h
        hT[i] = h
    y += skip * x
    out = {"y": (y * silu(z)).view(s["x"].shape), "final": hT}
    if not train:
        return out
    dy = s["dy"].to(f).reshape(-1, D)
    g = dy * silu(z)
    out.update(dz=(dy * y * dsilu(z)).view(s["x"].shape), dskip=(g * x).sum(0))
    dA, dh0 = torch.zeros(D, E, dtype=f, device=DEV), s["dhT"].to(f)
    ddt, SB, dB, dC = torch.empty_like(x), torch.empty_like(x), torch.empty_like(Bm), torch.empty_like(Cm)
    for i in range(n):
        S = dh0[i].clone()
        for k in range(cu[i + 1] - 1, cu[i] - 1, -1):
            S = torch.addcmul(by(S), g[k].view(G, -1, 1), Cm[k][:, None]).view(D, E)
            dC[k] = torch.bmm(g[k].view(G, 1, -1), by(kept[k]))[:, 0]
            dB[k] = torch.bmm(dx_in[k].view(G, 1, -1), by(S))[:, 0]
            SB[k] = torch.bmm(by(S), Bm[k][:, :, None]).view(D)
            S = S * torch.exp(dt[k][:, None] * A)
            q = S * (kept[k - 1] if k > cu[i] else h0[i])
            torch.addcmul(dA, q, dt[k][:, None], out=dA)
            ddt[k] = (q * A).sum(1)
        dh0[i] = S
    dpre = (ddt + x * SB) * torch.sigmoid(pre)
    out.update(dx=(skip * g + dt * SB).view(s["x"].shape), ddt=dpre.view(s["x"].shape), dbias=dpre.sum(0), dA=dA, d_initial=dh0,
               dB=dB.view(s["Bm"].shape), dC=dC.view(s["Cm"].shape))
    return out
