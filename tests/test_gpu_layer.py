"""A state space layer's operators together, as a model uses them: a block trained (norm, convolution,
scan and back), and the same block generating under beam search with its states in a cache."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_layer as pl
from gpu_util import BF, F, blank, cu_of, dev, gpu, ints, normal, same, say

pytestmark = pytest.mark.gpu

D, E, W, EPS = 96, 16, 4, 1e-6
BOUNDS = [0, 37, 37, 150, 290]
T, N = BOUNDS[-1], len(BOUNDS) - 1


def weights():
    g = torch.Generator().manual_seed(0)
    return {"norm": normal(g, (D,), std=0.2, mean=1.0), "conv": normal(g, (D, W), std=0.4), "cb": normal(g, (D,), std=0.1),
            "A": -torch.rand(D, E, generator=g) * 4 - 0.05, "skip": normal(g, (D,)), "bias": normal(g, (D,), mean=-2.0)}


def block(x, res, w, i, cu, n, carry=None):
    """norm of the residual stream -> convolution -> scan; everything that the way back needs."""
    new = lambda: blank(x.shape, x.dtype)  # noqa: E731
    o = {"h": new(), "res": new(), "c": new(), "y": new(), "rstd": blank((x.numel() // D,)), "cs": blank((n, W - 1, D)), "hs": blank((n, D, E))}
    kda.rmsnorm_fwd(x, w["norm"], EPS, o["h"], residual=res, residual_out=o["res"], rstd=o["rstd"])
    kda.conv_fwd(o["h"], w["conv"], w["cb"], o["c"], final_state=o["cs"], cu_seqlens=cu)
    kda.ssm_fwd(o["c"], i["dt"], w["A"], i["B"], i["C"], o["y"], D=w["skip"], z=i["z"], dt_bias=w["bias"], final_state=o["hs"], cu_seqlens=cu,
                carry=carry)
    return o


def inputs(T, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return {"x": normal(g, (1, T, D), dtype), "res": normal(g, (1, T, D), dtype), "dt": normal(g, (1, T, D), dtype, 0.7),
            "B": normal(g, (1, T, 1, E), dtype), "C": normal(g, (1, T, 1, E), dtype), "z": normal(g, (1, T, D), dtype),
            "dy": normal(g, (1, T, D), dtype), "dres": normal(g, (1, T, D), dtype)}


def test_training_step():
    """Forward and backward through the block in fp32, each operator's gradient from the one after it."""
    w, i = weights(), inputs(T, F, 1)
    gw, gi, cu = {k: gpu(t) for k, t in w.items()}, {k: gpu(t) for k, t in i.items()}, cu_of(BOUNDS)
    carry = blank(kda.ssm_carry_shape(1, T, D, E))
    o = block(gi["x"], gi["res"], gw, gi, cu, N, carry)
    new = lambda t: blank(t.shape, t.dtype)  # noqa: E731
    dc, ddt, dA, dB, dC, dz = new(o["c"]), new(o["c"]), new(gw["A"]), new(gi["B"]), new(gi["B"]), new(o["c"])
    dskip, dbias, dh, dcw, dcb, dx, dnorm = (new(t) for t in (gw["skip"], gw["bias"], o["h"], gw["conv"], gw["cb"], gi["x"], gw["norm"]))
    kda.ssm_bwd(o["c"], gi["dt"], gw["A"], gi["B"], gi["C"], gi["dy"], carry, dc, ddt, dA, dB, dC, D=gw["skip"], d_D=dskip, z=gi["z"], d_z=dz,
                dt_bias=gw["bias"], d_dt_bias=dbias, cu_seqlens=cu)
    kda.conv_bwd(o["h"], gw["conv"], gw["cb"], dc, dh, d_weight=dcw, d_bias=dcb, cu_seqlens=cu)
    kda.rmsnorm_bwd(dh, o["res"], gw["norm"], o["rstd"], dx, d_weight=dnorm, d_residual=gi["dres"])
    # the same by automatic differentiation in 64 bits
    f = torch.float64
    p = {k: t.to(f).requires_grad_() for k, t in w.items()}
    q = {k: t[0].to(f).requires_grad_() for k, t in i.items()}
    s = q["x"] + q["res"]
    h = s * (s.square().mean(1, keepdim=True) + EPS) ** -0.5 * p["norm"]
    ys = []
    for lo, hi in zip(BOUNDS[:-1], BOUNDS[1:]):
        v = torch.cat([torch.zeros(W - 1, D, dtype=f), h[lo:hi]])
        u = p["cb"] + sum(p["conv"][:, j] * v[j:j + hi - lo] for j in range(W))
        c = torch.nn.functional.silu(u)
        st = torch.zeros(D, E, dtype=f)
        for k in range(lo, hi):
            dt = torch.nn.functional.softplus(q["dt"][k] + p["bias"])
            st = torch.exp(dt[:, None] * p["A"]) * st + (dt * c[k - lo])[:, None] * q["B"][k, 0]
            ys.append((st @ q["C"][k, 0] + p["skip"] * c[k - lo]) * torch.nn.functional.silu(q["z"][k]))
    y = torch.stack(ys)
    ((y * q["dy"].detach()).sum() + (s * q["dres"].detach()).sum()).backward()
    say("block", float((o["y"][0].cpu() - y.detach()).abs().max()))
    for name, got, want in (("y", o["y"][0], y), ("dx", dx[0], q["x"].grad), ("dnorm", dnorm, p["norm"].grad), ("dconv", dcw, p["conv"].grad),
                            ("dcb", dcb, p["cb"].grad), ("dA", dA, p["A"].grad), ("dskip", dskip, p["skip"].grad), ("dbias", dbias, p["bias"].grad),
                            ("ddt", ddt[0], q["dt"].grad), ("dB", dB[0], q["B"].grad), ("dC", dC[0], q["C"].grad), ("dz", dz[0], q["z"].grad)):
        off = (got.cpu().double() - want.detach()).norm() / want.detach().norm()
        # some hundred roundings of 2^-24 in a row along a value's way, here added up as if all went one way
        assert float(off) <= 500 * 2.0 ** -24, (name, float(off))


def test_generation_under_beam_search():
    """Prompts through the block at once, then steps of beam search: every beam's states in the cache
    are those of its own tokens, run from the start."""
    beams, V, steps, prompts = 4, 50, 6, [9, 17, 1]
    w = {k: gpu(t) for k, t in weights().items()}
    g = torch.Generator().manual_seed(3)
    emb, head = gpu(normal(g, (V, D))), gpu(normal(g, (D, V), std=0.3))
    mix = {k: gpu(normal(g, (D, s), std=0.2)) for k, s in (("dt", D), ("B", E), ("C", E), ("z", D))}
    n = len(prompts)

    def side(t):   # a toy model's other inputs, from the tokens' embeddings
        x = emb[t]
        return {"x": x, "dt": x @ mix["dt"], "B": (x @ mix["B"])[..., None, :].contiguous(), "C": (x @ mix["C"])[..., None, :].contiguous(),
                "z": x @ mix["z"]}
    toks = [torch.randint(0, V, (k,), generator=g).tolist() for k in prompts]

    def whole(seqs):
        """Logits after the last token, and both states, of sequences of tokens."""
        cu = [0]
        for s in seqs:
            cu.append(cu[-1] + len(s))
        i = {k: t[None].contiguous() for k, t in side(torch.tensor(sum(seqs, []), device=dev())).items()}
        o = block(i["x"], None, w, i, cu_of(cu), len(seqs))
        return o["y"][0, [c - 1 for c in cu[1:]]] @ head, o["cs"], o["hs"]
    logits, cs, hs = whole(toks)
    S = n * beams + 2
    conv_pool, ssm_pool = torch.zeros(1, S, W - 1, D, device=dev()), torch.zeros(1, S, D, E, device=dev())
    used = ints([1] * n + [0] * (S - n))
    conv_pool[0, :n], ssm_pool[0, :n] = cs, hs
    src, dst = ints([k for k in range(n) for _ in range(beams - 1)]), ints([0] * (n * (beams - 1)))
    kda.cache_fork(ssm_pool, used, src, dst)
    kda.cache_copy(conv_pool, src, dst)
    slots = torch.cat([torch.arange(n, dtype=torch.int32, device=dev())[:, None], dst.view(n, beams - 1)], 1).contiguous()
    scores = torch.full((n, beams), float("-inf"), device=dev())
    scores[:, 0] = 0   # alike so far: one of them counts
    logits = logits[:, None].expand(n, beams, V).contiguous()
    history = [[list(t) for _ in range(beams)] for t in toks]
    for step in range(steps):
        tokens, parents, new_slots = (torch.empty(n, beams, dtype=torch.int32, device=dev()) for _ in range(3))
        new_scores = torch.empty_like(scores)
        kda.beam_select(logits, scores, tokens, parents, new_scores)
        for pool in (conv_pool, ssm_pool):
            kda.cache_reorder(pool, slots, parents, new_slots)
        slots, scores = new_slots, new_scores
        history = [[history[a][p] + [t] for p, t in zip(ps, ts)] for a, (ps, ts) in enumerate(zip(parents.tolist(), tokens.tolist()))]
        i = side(tokens.view(-1).long())
        h, c, y = blank((n * beams, D)), blank((n * beams, D)), blank((n * beams, D))
        at = slots.view(-1)
        kda.rmsnorm_fwd(i["x"], w["norm"], EPS, h)
        kda.conv_step(h, w["conv"], w["cb"], c, conv_pool[0], at, at)
        kda.ssm_step(c, i["dt"], w["A"], i["B"], i["C"], y, ssm_pool[0], at, at, D=w["skip"], z=i["z"], dt_bias=w["bias"])
        logits = (y @ head).view(n, beams, V)
        want, cs, hs = whole([s for row in history for s in row])
        # the same sums, grouped by tokens or by steps, in fp32
        torch.testing.assert_close(logits.view(-1, V), want, rtol=1e-4, atol=1e-4)
        torch.testing.assert_close(ssm_pool[0, at.long()], hs, rtol=1e-4, atol=1e-5)
        torch.testing.assert_close(conv_pool[0, at.long()], cs, rtol=1e-4, atol=1e-5)
    assert len({tuple(s) for s in history[0]}) == beams


def test_8_bit_output_of_the_norm_for_the_next_product():
    i = inputs(64, BF, 5)
    y8, sc = torch.empty(1, 64, D, device=dev(), dtype=torch.float8_e4m3fn), blank((1, 64, 1))
    y = blank((1, 64, D), BF)
    kda.rmsnorm_fwd(gpu(i["x"]), None, EPS, y8, residual=gpu(i["res"]), scales=sc)
    kda.rmsnorm_fwd(gpu(i["x"]), None, EPS, y, residual=gpu(i["res"]))
    a, b = y8.float() * sc, y.float()
    # half a step of 8 bits, 2^-4 of a value or 2^-10 of the scale, and of bf16
    assert bool(((a - b).abs() <= b.abs() * (2.0 ** -4 + 2.0 ** -7) + sc * 2.0 ** -10).all())
    assert not same(y, blank((1, 64, D), BF)) and pl.U == 2.0 ** -24


def test_one_workspace_for_the_largest_call_serves_smaller_ones():
    g = torch.Generator().manual_seed(5)
    W, V, k = 8, 8192, 8
    x, scores = gpu(normal(g, (64, W, V), BF, 3.0)), gpu(-torch.rand(64, W, generator=g))
    ws = torch.full((kda.beam_workspace_size(64, W, V, k),), 255, dtype=torch.uint8, device=dev())
    for N in (64, 63, 5, 1):
        out = []
        for w in (None, ws):
            t, p, s = (torch.zeros(N, k, dtype=d, device=dev()) for d in (torch.int32, torch.int32, F))
            kda.beam_select(x[:N], scores[:N], t, p, s, workspace=w)
            out.append((t, p, s))
        assert all(torch.equal(a, b) for a, b in zip(*out)), N
    T, D, E = 17000, 64, 4
    x, dt, dy, B, C = (gpu(normal(g, (1, T, d), BF)) for d in (D, D, D, E, E))
    A = gpu(-torch.rand(D, E, generator=g))
    wf, wb = (torch.full((kda.ssm_workspace_size(1, T, D, E, backward=b),), 255, dtype=torch.uint8, device=dev()) for b in (False, True))
    for n in (T, 16384, 8256, 8192, 8000, 64, 1):
        say("workspace", n)
        i = [t[:, :n].contiguous() for t in (x, dt, dy)] + [t[:, :n].unsqueeze(2).contiguous() for t in (B, C)]
        out = []
        for f, b in ((None, None), (wf, wb)):
            carry = blank(kda.ssm_carry_shape(1, n, D, E))
            o = [blank(i[0].shape, BF), blank(i[0].shape, BF), blank(i[0].shape, BF), blank(A.shape), blank(i[3].shape, BF), blank(i[3].shape, BF)]
            kda.ssm_fwd(i[0], i[1], A, i[3], i[4], o[0], carry=carry, workspace=f)
            kda.ssm_bwd(i[0], i[1], A, i[3], i[4], i[2], carry, *o[1:], workspace=b)
            out.append(o)
        assert all(same(a, b) for a, b in zip(*out)), n
