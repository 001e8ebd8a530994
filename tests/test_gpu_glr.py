"""Gated linear recurrence on the GPU against its 64-bit form, forward, backward and single
tokens on a cache's slots: types, odd widths, lengths around a tile's, empty sequences, gates
that start over, tokens of no sequence, states written over, graphs, streams."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_ops as po

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def say(*a):
    print("[gpu-test]", *a, flush=True)


class Case:
    def __init__(self, dtype, D, B=1, T=None, lengths=None, state=None, seed=0, gate=1.0, lead=0, tail=0):
        gen = torch.Generator().manual_seed(seed)
        cu = None
        if lengths is not None:
            cu = [lead]
            for n in lengths:
                cu.append(cu[-1] + n)
            T = cu[-1] + tail
        self.B, self.T, self.D, self.dtype = B, T, D, dtype
        self.cu = None if cu is None else torch.tensor(cu, dtype=torch.int64)
        self.n = B if cu is None else len(lengths)
        r = lambda *s: torch.randn(*s, generator=gen)
        self.x, self.dy = r(B, T, D).to(dtype), r(B, T, D).to(dtype)
        self.g = (-torch.exp(r(B, T, D) * 1.2 - 2.5) * gate).to(dtype)
        self.h0 = None if state is None else r(self.n, D).to(state)
        self.dhT = r(self.n, D)
        self.state = state
        self.sp = po.spans(cu, B, T)

    def gpu(self, name):
        t = getattr(self, name)
        return None if t is None else t.to(dev())

    def plain(self):
        flat = lambda t: t.reshape(-1, self.D)
        return po.glr(flat(self.x), flat(self.g), self.sp, self.h0, flat(self.dy), self.dhT)

    def run(self, bwd=True, fill=float("nan")):
        d = dev()
        x, g, cu, h0 = self.gpu("x"), self.gpu("g"), self.gpu("cu"), self.gpu("h0")
        new = lambda: torch.full((self.B, self.T, self.D), fill, dtype=self.dtype, device=d)
        out = {"y": new(), "final": torch.full((self.n, self.D), fill, dtype=self.state or F, device=d),
               "carry": torch.full(kda.glr_carry_shape(self.B, self.T, self.D), fill, device=d)}
        kda.glr_fwd(x, g, out["y"], initial_state=h0, final_state=out["final"], cu_seqlens=cu, carry=out["carry"])
        if bwd:
            out.update(dx=new(), dg=new(), d_initial=torch.full((self.n, self.D), fill, device=d))
            kda.glr_bwd(x, g, self.gpu("dy"), out["carry"], out["dx"], out["dg"], initial_state=h0,
                        d_final=self.gpu("dhT"), d_initial=out["d_initial"], cu_seqlens=cu)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        v, e = self.plain()
        D = self.D
        for k in ("y", "dx", "dg"):
            po.assert_near(k, out[k].reshape(-1, D), v[k], e[k])
        for k in ("final", "d_initial"):
            po.assert_near(k, out[k], v[k], e[k])
        inside = [t for t in range(0, self.B * self.T, 128) if any(b < t < t1 for b, t1 in self.sp)]
        rows = [t // 128 for t in inside]
        po.assert_near("carry", out["carry"][rows], v["before"][inside], e["before"][inside])


LENGTHS = [[1], [0, 1, 0, 0, 2], [127, 129], [128, 128], [130, 0, 1, 255, 256, 3], [700], [1] * 300, [0, 0]]


@pytest.mark.parametrize("dtype", [BF, HF, F], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [1, 7, 64, 136, 1000])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "-".join(map(str, v[:6])) + f"x{len(v)}")
def test_packed(dtype, D, lengths):
    say("packed", dtype, D, lengths[:8])
    state = [None, F, BF][(D + len(lengths)) % 3]
    c = Case(dtype, D, lengths=lengths, state=state, seed=D)
    c.check(c.run())


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 5), (3, 1, 64), (2, 100, 24), (3, 128, 129), (2, 129, 8), (4, 300, 257), (1, 2000, 40),
                                   (5, 17, 1), (1, 4100, 512)])
def test_rows(dtype, B, T, D):
    say("rows", dtype, B, T, D)
    c = Case(dtype, D, B=B, T=T, state=[F, None, BF][T % 3], seed=T)
    c.check(c.run())


@pytest.mark.parametrize("gate", [0.0, 1e-4, 100.0], ids=["none", "slow", "fast"])
def test_gates(gate):
    """No decay at all (a running sum), hardly any, and states forgotten at once."""
    say("gate", gate)
    c = Case(F, 72, lengths=[500, 3, 200], state=F, gate=gate, seed=3)
    c.check(c.run())


def test_gates_that_start_over():
    """-inf forgets everything before, at a sequence's first token the initial state too; its
    gradient, and the state's before it, is zero."""
    say("gates of -inf")
    c = Case(BF, 40, lengths=[300, 129, 1, 5], state=F, seed=4)
    for t in (0, 5, 127, 128, 200, 299, 300, 429):
        c.g[0, t] = float("-inf")
    c.g[0, 64, ::3] = float("-inf")
    out = c.run()
    c.check(out)
    assert float(out["dg"][0, 5].abs().max()) == 0.0 and float(out["d_initial"][0].abs().max()) == 0.0


def test_positive_gates_and_no_clamp():
    say("gates above zero")
    c = Case(F, 33, B=2, T=150, state=F, seed=5)
    c.g[:, ::2] = 0.05
    c.check(c.run())


def test_nan_and_inf_stay_in_their_channel_and_sequence():
    say("NaN and infinities in some places")
    c = Case(F, 24, lengths=[200, 150, 140], state=F, seed=6)
    clean = c.run()
    c.x[0, 210, 3] = float("nan")
    c.x[0, 260, 7] = float("inf")
    c.dy[0, 300, 9] = float("nan")
    out = c.run()
    for k in ("y", "dx", "dg"):
        t = out[k][0].cpu()
        assert torch.equal(t[:200], clean[k][0, :200].cpu()) and torch.equal(t[350:], clean[k][0, 350:].cpu()), k
        keep = [d for d in range(24) if d not in (3, 7, 9)]
        assert torch.equal(t[:, keep], clean[k][0].cpu()[:, keep]), k
    y = out["y"][0].cpu()
    assert torch.isnan(y[210:350, 3]).all() and torch.isinf(y[260, 7]) and torch.isfinite(y[200:210, 3]).all()


@pytest.mark.parametrize("lead,tail", [(0, 70), (5, 0), (130, 300)])
@pytest.mark.parametrize("D", [16, 9])
def test_tokens_of_no_sequence(lead, tail, D):
    """Tokens before the first sequence and behind the last are neither read nor written."""
    say("tokens of no sequence", lead, tail, D)
    c = Case(BF, D, lengths=[100, 0, 150], state=F, lead=lead, tail=tail, seed=7)
    end = lead + 250
    for t in (c.x, c.g, c.dy):
        t[0, :lead] = float("nan")
        t[0, end:] = float("nan")
    out = c.run(fill=-3.0)
    v, e = po.glr(torch.nan_to_num(c.x[0]), torch.nan_to_num(c.g[0]), c.sp, c.h0, torch.nan_to_num(c.dy[0]), c.dhT)
    for k in ("y", "dx", "dg"):
        got = out[k][0]
        assert (got[:lead] == -3).all() and (got[end:] == -3).all(), k
        po.assert_near(k, got[lead:end], v[k][lead:end], e[k][lead:end])
    for k in ("final", "d_initial"):
        po.assert_near(k, out[k], v[k], e[k])


@pytest.mark.parametrize("kw", [dict(B=3, T=300), dict(lengths=[1, 200, 0, 128, 64]), dict(B=2, T=3), dict(lengths=[1, 1, 0])],
                         ids=["rows", "packed", "short", "tokens"])
@pytest.mark.parametrize("state", [F, BF], ids=["fp32", "bf16"])
def test_state_written_over(kw, state):
    """final_state may be initial_state: the same bits as with two buffers."""
    say("state in place", kw, state)
    c = Case(BF, 136, state=state, seed=8, **kw)
    ref = c.run(bwd=False)
    st, y = c.gpu("h0"), torch.empty_like(ref["y"])
    kda.glr_fwd(c.gpu("x"), c.gpu("g"), y, initial_state=st, final_state=st, cu_seqlens=c.gpu("cu"))
    assert torch.equal(st, ref["final"]) and torch.equal(y, ref["y"])


def test_chained_calls_equal_one():
    """A prefix and the rest, the state passed between them, against the call on all tokens."""
    say("two calls chained through the state")
    c = Case(F, 64, B=2, T=700, state=F, seed=9)
    v, e = c.plain()
    x, g, st = c.gpu("x"), c.gpu("g"), c.gpu("h0")
    ys = []
    for a, b in ((0, 1), (1, 300), (300, 700)):
        y = torch.empty(2, b - a, 64, device=dev())
        kda.glr_fwd(x[:, a:b].contiguous(), g[:, a:b].contiguous(), y, initial_state=st, final_state=st)
        ys.append(y)
    po.assert_near("y", torch.cat(ys, 1).reshape(-1, 64), v["y"], e["y"])
    po.assert_near("final", st, v["final"], e["final"])


def test_no_tokens():
    say("T = 0")
    e = torch.empty(2, 0, 24, dtype=BF, device=dev())
    h0, fin, dh = torch.randn(2, 24, device=dev()), torch.empty(2, 24, device=dev()), torch.empty(2, 24, device=dev())
    carry = torch.empty(0, 24, device=dev())
    kda.glr_fwd(e, e, e, initial_state=h0, final_state=fin, carry=carry)
    kda.glr_bwd(e, e, e, carry, e, e, initial_state=h0, d_final=h0, d_initial=dh)
    assert torch.equal(fin, h0) and torch.equal(dh, h0)
    kda.glr_fwd(e, e, e, final_state=fin)
    assert float(fin.abs().max()) == 0.0


def test_gradients_against_differences():
    """Directional differences of the 64-bit forward pass. The loss is linear in x and h0 (any
    step will do), and smooth in g: a central difference of step h is off by h^2/6 of the third
    derivative along the direction; with h = 1e-3 and |direction| <= 3 per gate and memories of
    at most 40 tokens that is below 1e-6 * (3 * 40)^3 / 6 = 0.3 of the absolute sum, so the
    step is taken at 1e-5: below 3e-5 of it, beside 1e-16 / 1e-5 of cancellation."""
    say("gradients against differences")
    c = Case(F, 12, lengths=[40, 0, 17], state=F, seed=10)
    out = c.run()
    gen = torch.Generator().manual_seed(1)
    f = torch.float64
    dirs = {k: torch.randn(t.shape, generator=gen).clamp(-3, 3).to(f) for k, t in (("x", c.x[0]), ("g", c.g[0]), ("h0", c.h0))}

    def loss(name, step):
        v = {"x": c.x[0].to(f), "g": c.g[0].to(f), "h0": c.h0.to(f)}
        v[name] = v[name] + step * dirs[name]
        r, _ = po.glr(v["x"], v["g"], c.sp, v["h0"])
        return (r["y"] * c.dy[0].to(f)).sum() + (r["final"] * c.dhT.to(f)).sum()

    for name, grad in (("x", out["dx"][0]), ("g", out["dg"][0]), ("h0", out["d_initial"])):
        want = (loss(name, 1e-5) - loss(name, -1e-5)) / 2e-5
        terms = grad.cpu().to(f) * dirs[name]
        assert abs(terms.sum() - want) <= 1e-4 * terms.abs().sum(), name


def test_same_bits_again():
    say("the same call gives the same bits")
    c = Case(BF, 1024, lengths=[1000, 1, 3000, 77, 0, 900], state=F, seed=11)
    a = c.run()
    for _ in range(3):
        b = c.run()
        for k in ("y", "final", "dx", "dg", "d_initial"):
            assert torch.equal(a[k], b[k]), k


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last channels of the last tokens against a call on those
    channels alone (a channel's values do not depend on the others)."""
    say("offsets past 2^31 elements")
    T, D, W = 8200, 262144 + 64, 64
    d = dev()
    gen = torch.Generator(device=d).manual_seed(0)
    x = torch.randn(1, T, D, generator=gen, device=d, dtype=BF)
    g = -torch.rand(1, T, D, generator=gen, device=d, dtype=BF)
    assert x.numel() > 2 ** 31
    y, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    fin, carry = torch.empty(1, D, device=d), torch.empty(kda.glr_carry_shape(1, T, D), device=d)
    kda.glr_fwd(x, g, y, final_state=fin, carry=carry)
    kda.glr_bwd(x, g, x, carry, dx, dg)
    xs, gs = x[..., -W:].contiguous(), g[..., -W:].contiguous()
    ys, dxs, dgs = torch.empty_like(xs), torch.empty_like(xs), torch.empty_like(xs)
    fs, cs = torch.empty(1, W, device=d), torch.empty(kda.glr_carry_shape(1, T, W), device=d)
    kda.glr_fwd(xs, gs, ys, final_state=fs, carry=cs)
    kda.glr_bwd(xs, gs, xs, cs, dxs, dgs)
    assert torch.equal(y[..., -W:], ys) and torch.equal(fin[:, -W:], fs)
    assert torch.equal(dx[..., -W:], dxs) and torch.equal(dg[..., -W:], dgs)


@pytest.mark.parametrize("dtype", [BF, HF, F], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("state", [F, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 129), (7, 64), (33, 1024)])
def test_step(dtype, state, N, D):
    """Slots of their own, of several sequences, none (zeros, not written), and the rest of the
    cache left as it was."""
    say("step", dtype, state, N, D)
    gen = torch.Generator().manual_seed(N)
    S = 2 * N + 3
    pool = torch.randn(S, D, generator=gen).to(state)
    x, g = torch.randn(N, D, generator=gen).to(dtype), -torch.rand(N, D, generator=gen).to(dtype)
    perm = torch.randperm(S, generator=gen)
    src, dst = perm[:N].to(torch.int32), perm[N:2 * N].to(torch.int32)
    if N > 2:
        src[1], src[2], dst[0] = -1, src[0], S
        src[N - 1] = S + 5
    if N > 6:
        dst[4] = src[4]   # in place
    h0 = torch.stack([pool[i].float() if 0 <= i < S else torch.zeros(D) for i in src.tolist()])
    v, e = po.glr(x, g, [(i, i + 1) for i in range(N)], h0)
    p, y = pool.to(dev()), torch.full((N, D), float("nan"), dtype=dtype, device=dev())
    kda.glr_step(x.to(dev()), g.to(dev()), y, p, src.to(dev()), dst.to(dev()))
    po.assert_near("y", y, v["y"], e["y"])
    kept = torch.ones(S, dtype=torch.bool)
    for i, s in enumerate(dst.tolist()):
        if 0 <= s < S:
            kept[s] = False
            po.assert_near("state", p[s], v["final"][i], e["final"][i])
    assert torch.equal(p.cpu()[kept], pool[kept])


def test_step_of_no_sequence():
    e = torch.empty(0, 8, device=dev())
    i = torch.empty(0, dtype=torch.int32, device=dev())
    pool = torch.ones(2, 8, device=dev())
    kda.glr_step(e, e, e, pool, i, i)
    assert (pool == 1).all()


def test_graph_replays():
    """A training step captured once and replayed with new inputs, with eager calls between,
    and a second graph that uses the same workspace."""
    say("graphs of forward and backward, one workspace")
    c = Case(BF, 264, lengths=[300, 0, 129, 700, 5], state=F, seed=12)
    x, g, dy, cu, h0, dhT = (c.gpu(k) for k in ("x", "g", "dy", "cu", "h0", "dhT"))
    ws = torch.empty(max(1, kda.glr_workspace_size(1, c.T, 264, c.n)), dtype=torch.uint8, device=dev())

    def buffers():
        return {"y": torch.empty_like(x), "f": torch.empty_like(h0), "dx": torch.empty_like(x), "dg": torch.empty_like(x),
                "d0": torch.empty_like(h0), "c": torch.empty(kda.glr_carry_shape(1, c.T, 264), device=dev())}

    def step(o):
        kda.glr_fwd(x, g, o["y"], initial_state=h0, final_state=o["f"], cu_seqlens=cu, carry=o["c"], workspace=ws)
        kda.glr_bwd(x, g, dy, o["c"], o["dx"], o["dg"], initial_state=h0, d_final=dhT, d_initial=o["d0"], cu_seqlens=cu,
                    workspace=ws)

    outs, graphs = [buffers(), buffers()], []
    side = torch.cuda.Stream(dev())
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(outs[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for o in outs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(o)
        graphs.append(gr)
    for seed in (1, 2, 3):
        n = Case(BF, 264, lengths=[300, 0, 129, 700, 5], state=F, seed=20 + seed)
        for t, k in ((x, "x"), (g, "g"), (dy, "dy"), (h0, "h0"), (dhT, "dhT")):
            t.copy_(getattr(n, k))
        for o, gr in zip(outs, graphs):
            gr.replay()
        eager = buffers()
        step(eager)
        graphs[0].replay()
        torch.cuda.synchronize()
        for o in outs:
            for k in ("y", "f", "dx", "dg", "d0"):
                assert torch.equal(o[k], eager[k]), f"seed {seed}: {k}"


def test_streams_at_once():
    """Calls on three streams, each with its own workspace from the allocator, against each alone."""
    say("three streams")
    cs = [Case(BF, 512, lengths=[2000, 5, 900], state=F, seed=13), Case(F, 100, B=3, T=777, seed=14),
          Case(HF, 2048, B=1, T=1500, state=BF, seed=15)]
    refs = [c.run() for c in cs]
    streams = [torch.cuda.Stream(dev()) for _ in cs]
    for _ in range(3):
        got = []
        args = [{k: c.gpu(k) for k in ("x", "g", "dy", "cu", "h0", "dhT")} for c in cs]
        outs = [{k: torch.zeros_like(v) for k, v in r.items()} for r in refs]
        torch.cuda.synchronize()
        for c, a, o, st in zip(cs, args, outs, streams):
            with torch.cuda.stream(st):
                kda.glr_fwd(a["x"], a["g"], o["y"], initial_state=a["h0"], final_state=o["final"], cu_seqlens=a["cu"], carry=o["carry"])
                kda.glr_bwd(a["x"], a["g"], a["dy"], o["carry"], o["dx"], o["dg"], initial_state=a["h0"], d_final=a["dhT"],
                            d_initial=o["d_initial"], cu_seqlens=a["cu"])
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            for k in ("y", "final", "dx", "dg", "d_initial"):
                assert torch.equal(o[k], r[k]), k


def test_boundaries_out_of_order_stay_in_bounds():
    """Boundaries that break the precondition give unspecified results inside the buffers only;
    what lies around them is left."""
    say("bad boundaries")
    d = dev()
    T, D = 300, 40
    room = torch.full((T + 64, D), 7.0, device=d)
    for cu in ([0, 500, 300], [-5, 100, 90], [10, 5, 400], [0, 1 << 40, -(1 << 40)]):
        y = room.clone()
        x = torch.randn(1, T, D, device=d)
        st = torch.zeros(2, D, device=d)
        kda.glr_fwd(x, -x.abs(), y[32:32 + T].unsqueeze(0), final_state=st, cu_seqlens=torch.tensor(cu, device=d))
        torch.cuda.synchronize()
        assert (y[:32] == 7).all() and (y[32 + T:] == 7).all()


@pytest.mark.parametrize("N,T", [(70000, 70000), (70000, 200000)])
def test_many_sequences(N, T):
    """More sequences than a launch's second grid dimension holds, by tokens and by tiles."""
    say("sequences", N, "tokens", T)
    gen = torch.Generator().manual_seed(0)
    cut = torch.sort(torch.randint(0, T + 1, (N - 1,), generator=gen)).values
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.full((1,), T)])
    D = 8
    x, g = torch.randn(1, T, D, generator=gen), -torch.rand(1, T, D, generator=gen)
    h0 = torch.randn(N, D, generator=gen)
    y, fin = torch.empty(1, T, D, device=dev()), torch.empty(N, D, device=dev())
    kda.glr_fwd(x.to(dev()), g.to(dev()), y, initial_state=h0.to(dev()), final_state=fin, cu_seqlens=cu.to(dev()))
    # the recurrence over all sequences at once, token i of each (none is longer than the longest)
    f = torch.float64
    lengths = cu[1:] - cu[:-1]
    h, e, s = h0.to(f), torch.zeros(N, D, dtype=f), h0.to(f).abs()
    yv, ye = torch.zeros(T, D, dtype=f), torch.zeros(T, D, dtype=f)
    for i in range(int(lengths.max())):
        on = (lengths > i).nonzero()[:, 0]
        t = cu[on] + i
        a = g[0, t].to(f).exp()
        h[on] = a * h[on] + x[0, t].to(f)
        s[on] = a * s[on] + x[0, t].to(f).abs()
        e[on] = a * e[on] + (8 + 2 * g[0, t].to(f).abs()) * po.U * s[on]
        yv[t], ye[t] = h[on], e[on]
    po.assert_near("y", y[0], yv, ye)
    po.assert_near("final", fin, h, e)


def test_validation_of_boundaries(monkeypatch):
    """KDA_VALIDATE=1: contents that break the precondition are refused, nothing is written."""
    say("KDA_VALIDATE")
    monkeypatch.setenv("KDA_VALIDATE", "1")
    d = dev()
    x = torch.randn(1, 40, 16, device=d)
    y = torch.full_like(x, 7.0)
    carry, h = torch.zeros(kda.glr_carry_shape(1, 40, 16), device=d), torch.zeros(2, 16, device=d)
    for cu in ([0, 30, 20], [1, 20, 40], [0, 20, 39]):
        c = torch.tensor(cu, device=d)
        with pytest.raises(kda.KDAError) as e:
            kda.glr_fwd(x, -x.abs(), y, final_state=h, cu_seqlens=c)
        assert e.value.code == 4
        with pytest.raises(kda.KDAError) as e:
            kda.glr_bwd(x, -x.abs(), x, carry, y, y.clone(), cu_seqlens=c)
        assert e.value.code == 4
    assert (y == 7).all()
    kda.glr_fwd(x, -x.abs(), y, final_state=h, cu_seqlens=torch.tensor([0, 15, 40], device=d))


def test_refusals_of_the_wrappers():
    """Shapes, types, strides and devices that do not fit, before anything is launched."""
    d = dev()
    x, i = torch.zeros(2, 40, 16, device=d), torch.zeros(2, dtype=torch.int32, device=d)
    g, y, st = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(2, 16, device=d)
    carry = torch.zeros(1, 16, device=d)
    bad = [lambda: kda.glr_fwd(x, g.bfloat16(), y), lambda: kda.glr_fwd(x, g[:, :39], y), lambda: kda.glr_fwd(x, g, y[..., :15]),
           lambda: kda.glr_fwd(x.transpose(0, 1), g.transpose(0, 1), y.transpose(0, 1)), lambda: kda.glr_fwd(x, g.cpu(), y),
           lambda: kda.glr_fwd(x.double(), g.double(), y.double()), lambda: kda.glr_fwd(x, g, y, initial_state=st[:1]),
           lambda: kda.glr_fwd(x, g, y, initial_state=st, final_state=st.bfloat16()),
           lambda: kda.glr_fwd(x, g, y, cu_seqlens=torch.tensor([0, 80], device=d)),
           lambda: kda.glr_fwd(x, g, y, carry=carry.bfloat16()), lambda: kda.glr_bwd(x, g, x, carry[:, :8], y, g),
           lambda: kda.glr_bwd(x, g, x, carry, y, g.clone(), d_final=st.half()),
           lambda: kda.glr_step(x[0], g[0], y[0], st, i, i), lambda: kda.glr_step(x[0, :2], g[0, :2], y[0, :2], st, i.long(), i)]
    for n, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", n)
    with pytest.raises(kda.KDAError) as e:   # a view that starts between two 16-byte addresses
        flat = torch.zeros(2 * 40 * 16 + 1, device=d)
        kda.glr_fwd(flat[1:].view(2, 40, 16), g, y)
    assert e.value.code == 5
    with pytest.raises(kda.KDAError) as e:
        kda.glr_fwd(x, g, y, workspace=torch.empty(16, dtype=torch.uint8, device=d))
    assert e.value.code == 6


def test_waits_end(monkeypatch):
    """With no polls allowed every wait ends at once: values that had to be waited for are NaN,
    nothing else is written, and the next call is as ever."""
    say("waits cut short")
    c = Case(F, 192, lengths=[3000, 5, 2000], state=F, seed=16)
    ref = c.run()
    monkeypatch.setenv("KDA_GLR_POLLS", "0")
    cut = c.run()
    for k in ("y", "dx", "dg"):
        v, r = cut[k], ref[k]
        assert bool(((v == r) | torch.isnan(v)).all()), k
    assert torch.equal(cut["y"][0, :128], ref["y"][0, :128]) and torch.equal(cut["dx"][0, -1], ref["dx"][0, -1])
    monkeypatch.delenv("KDA_GLR_POLLS")
    again = c.run()
    for k in ref:
        assert torch.equal(torch.nan_to_num(again[k]), torch.nan_to_num(ref[k])), k


@pytest.mark.parametrize("gate", [1.0, 40.0, 400.0], ids=["usual", "strong", "strongest"])
@pytest.mark.parametrize("dtype", [F, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("kw", [dict(lengths=[5, 3000, 200]), dict(B=2, T=2500)], ids=["packed", "rows"])
def test_infinite_states_stay_infinite(kw, dtype, gate):
    """exp(g) of a gate from -87 on is above zero, however many are multiplied: an infinite state
    stays so to its sequence's end, and an infinite gradient to its first token."""
    say("infinite states", kw, dtype, gate)
    c = Case(dtype, 24, state=F, seed=17, **kw)
    c.g = (c.g.float() * gate).clamp(min=-87.0).to(dtype)
    clean = c.run()
    flat = lambda t: t.view(-1, 24)
    b, e = c.sp[1]
    flat(c.x)[b + 100, 3] = float("inf")
    flat(c.x)[b + 1111, 4] = float("-inf")
    c.h0[1, 5] = float("inf")
    flat(c.dy)[e - 200, 9] = float("inf")
    c.dhT[1, 10] = float("-inf")
    out = c.run()
    inf = float("inf")
    y, dx = out["y"].view(-1, 24).cpu(), out["dx"].view(-1, 24).cpu()
    assert (y[b + 100:e, 3] == inf).all() and (y[b + 1111:e, 4] == -inf).all() and (y[b:e, 5] == inf).all()
    assert out["final"][1, 3:6].tolist() == [inf, -inf, inf]
    assert (dx[b:e - 199, 9] == inf).all() and (dx[b:e, 10] == -inf).all()
    assert out["d_initial"][1, 9:11].tolist() == [inf, -inf]
    assert torch.equal(y[b:b + 100, 3], clean["y"].view(-1, 24)[b:b + 100, 3].cpu())
    keep = [d for d in range(24) if d not in (3, 4, 5, 9, 10)]
    for k in ("y", "dx", "dg"):
        t, r = out[k].view(-1, 24).cpu(), clean[k].view(-1, 24).cpu()
        assert torch.equal(t[:, keep], r[:, keep]) and torch.equal(t[:b], r[:b]) and torch.equal(t[e:], r[e:]), k
    # h_{t-1} is infinite and nothing that multiplies it is zero
    grad, h = out["dg"].view(-1, 24).cpu(), clean["dx"].view(-1, 24).cpu()
    some = h[b + 101:e, 3].float().abs() > 1e-30
    if gate == 1.0:
        assert torch.isinf(grad[b + 101:e, 3][some]).all()


@pytest.mark.parametrize("low", ["-inf", "lowest", "-88"])
@pytest.mark.parametrize("dtype", [F, BF, HF], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kw", [dict(lengths=[900, 40]), dict(lengths=[512, 30, 300]), dict(B=2, T=470), dict(B=1, T=30),
                                dict(lengths=[2, 1, 1, 1, 1, 2, 1])], ids=["packed", "tile", "rows", "few", "tokens"])
@pytest.mark.parametrize("D", [40, 41])
def test_starting_over_forgets_nan_and_infinities(D, kw, dtype, low):
    """A gate whose exponential is below 2^-126 (-87.4 and less, a type's lowest value and -inf
    among them) starts over from x_t whatever the state before it was, and no gradient passes it:
    the tokens after it, the gradients of those before it, and the initial state's, have the
    bits of a clean run."""
    say("starting over", D, kw, dtype, low)
    low = {"-inf": float("-inf"), "lowest": torch.finfo(dtype).min, "-88": -88.0}[low]
    c = Case(dtype, D, state=F, seed=18, **kw)
    where = []
    for b, e in c.sp:
        where.append(sorted({b, b + (e - b) // 2, e - 1}) if e - b > 2 else [e - 1])
    for ts in where:
        for t in ts:
            c.g.view(-1, D)[t] = low
    clean = c.run()
    c.h0[:, 1::3] = float("nan")
    c.h0[:, 2::6] = float("inf")
    for (b, e), ts in zip(c.sp, where):
        if e - b > 8:   # garbage between the gates
            c.x.view(-1, D)[ts[1] - 3, ::3] = float("nan")
            c.x.view(-1, D)[ts[2] - 3, 1::3] = float("-inf")
            c.dy.view(-1, D)[ts[1] + 2, ::2] = float("nan")
            c.dy.view(-1, D)[ts[2] - 1, 1::2] = float("inf")
    out = c.run()
    v = {k: t.reshape(-1, D).cpu() for k, t in out.items()}
    r = {k: t.reshape(-1, D).cpu() for k, t in clean.items()}
    for i, ((b, e), ts) in enumerate(zip(c.sp, where)):
        assert torch.equal(v["final"][i], r["final"][i])
        if ts[0] == b:
            assert (v["d_initial"][i] == 0).all()
        for t in ts:
            assert (v["dg"][t] == 0).all()
            assert torch.equal(v["y"][t], r["y"][t])
        if e - b > 8:
            half = ts[1]
            assert torch.equal(v["y"][half:ts[2] - 3], r["y"][half:ts[2] - 3])
            assert torch.equal(v["dx"][b:half], r["dx"][b:half])
            assert torch.equal(v["dg"][half + 1:ts[2] - 3].isnan(), v["dx"][half + 1:ts[2] - 3].isnan())
            assert v["y"][half - 3:half, ::3].isnan().all() and torch.isfinite(v["y"][half:ts[2] - 3]).all()
            assert v["dx"][half:half + 3, ::2].isnan().all()


@pytest.mark.parametrize("sign", [1.0, -1.0], ids=["nan", "-nan"])
@pytest.mark.parametrize("dtype", [F, BF, HF], ids=["fp32", "bf16", "fp16"])
def test_nan_gates_stop_at_a_start_over(dtype, sign):
    """A NaN gate, of either sign, reaches no token before or after a gate that starts over."""
    say("NaN gates", dtype, sign)
    c = Case(dtype, 16, lengths=[300], state=F, seed=19)
    for t in (41, 47, 200):
        c.g[0, t] = float("-inf")
    clean = c.run()
    bits = {F: torch.int32, BF: torch.int16, HF: torch.int16}[dtype]
    nan = torch.full((16,), float("nan")).to(dtype).view(bits) | 1
    low = torch.iinfo(bits).min
    c.g[0, 44] = (nan & torch.iinfo(bits).max if sign > 0 else nan | low).view(dtype)
    out = c.run()
    v, r = ({k: t.reshape(-1, 16).cpu() for k, t in o.items()} for o in (out, clean))
    for k, first, last in (("y", 44, 46), ("dx", 41, 43), ("dg", 42, 46)):
        assert v[k][first:last + 1].isnan().all(), k
        assert torch.equal(v[k][:first], r[k][:first]) and torch.equal(v[k][last + 1:], r[k][last + 1:]), k
    assert torch.equal(v["final"], r["final"]) and torch.equal(v["d_initial"], r["d_initial"])



def test_step_starts_over():
    say("a step that starts over")
    d = dev()
    pool = torch.full((3, 16), float("nan"), device=d)
    x, g = torch.randn(3, 16, device=d), torch.full((3, 16), float("-inf"), device=d)
    y = torch.empty_like(x)
    i = torch.arange(3, dtype=torch.int32, device=d)
    kda.glr_step(x, g, y, pool, i, i)
    assert torch.equal(y, x) and torch.equal(pool, x)
    pool.fill_(float("inf"))
    kda.glr_step(x, torch.full_like(x, -87.0), y, pool, i, i)
    assert (y == float("inf")).all()


@pytest.mark.parametrize("value", ["", "many", "12x", "-1", "4294967296", "99999999999999999999999"])
def test_a_cap_on_polls_that_is_no_number(monkeypatch, value):
    """KDA_GLR_POLLS that is not a whole number is not set, and one past 32 bits is the most
    there can be: waits go on."""
    say("KDA_GLR_POLLS", repr(value))
    c = Case(F, 192, lengths=[3000, 5, 2000], state=F, seed=16)
    ref = c.run()
    monkeypatch.setenv("KDA_GLR_POLLS", value)
    out = c.run()
    for k in ("y", "final", "dx", "dg", "d_initial"):
        assert torch.equal(out[k], ref[k]), k


@pytest.mark.parametrize("N,T", [(4096, 8192), (2000, 4000)])
def test_one_long_sequence_among_many_places(N, T):
    """A packed batch of few tokens a sequence on average, all of them in one: 0.2 ms are ten times
    what its tiles take, and a quarter of walking 4000 tokens one after the other."""
    say("one long sequence among", N)
    d = dev()
    x, g = torch.randn(1, T, 64, device=d), -torch.rand(1, T, 64, device=d)
    cu = torch.tensor([0] * (N // 2) + [T] * (N // 2 + 1), device=d)
    y, fin = torch.empty_like(x), torch.empty(N, 64, device=d)
    one, last = torch.empty_like(x), torch.empty(1, 64, device=d)
    kda.glr_fwd(x, g, one, final_state=last)
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        kda.glr_fwd(x, g, y, final_state=fin, cu_seqlens=cu)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert torch.equal(y, one) and torch.equal(fin[N // 2 - 1], last[0])
    assert min(times) < 0.2, times
