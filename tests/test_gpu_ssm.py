"""The selective state space scan on the GPU against its plain 64-bit form."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_layer as pl
from gpu_util import BF, DTYPES, F, H16, blank, covered, cu_of, dev, gpu, ints, normal, same, say, spans_of, untouched

pytestmark = pytest.mark.gpu

RAGGED = [0, 1, 1, 17, 20, 81, 145, 145, 210]
# B, T, D, E, G, bounds
SHAPES = [(1, 1, 1, 1, 1, None), (2, 5, 7, 3, 1, None), (1, 64, 64, 16, 1, None), (1, 65, 66, 16, 2, None), (3, 130, 24, 8, 3, None),
          (1, 200, 130, 16, 1, None), (1, 100, 40, 33, 1, None), (2, 70, 35, 20, 5, None), (1, 300, 16, 64, 1, None),
          (1, 210, 72, 16, 1, RAGGED), (1, 210, 33, 13, 1, RAGGED), (1, 210, 20, 40, 2, RAGGED), (1, 210, 130, 6, 1, RAGGED),
          (1, 150, 12, 16, 1, [9, 30, 30, 31, 140]), (3, 0, 8, 4, 1, None), (1, 0, 8, 4, 1, [0, 0]), (1, 128, 128, 16, 1, [0, 64, 128]),
          (1, 400, 20, 16, 1, [200, 201, 330]), (1, 300, 70, 8, 1, [0, 10, 64]), (1, 90, 300, 4, 4, [0, 0, 90]),
          (1, 70, 6, 2, 6, None)]


def make(B, T, D, E, G, bounds, dtype, state, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = len(bounds) - 1 if bounds else B
    i = {"x": normal(g, (B, T, D), dtype), "dt": normal(g, (B, T, D), dtype, 0.7), "A": -torch.rand(D, E, generator=g) * 4 - 0.05,
         "B": normal(g, (B, T, G, E), dtype), "C": normal(g, (B, T, G, E), dtype), "skip": normal(g, (D,)),
         "z": normal(g, (B, T, D), dtype), "bias": normal(g, (D,), mean=-2.0), "dy": normal(g, (B, T, D), dtype)}
    i["h0"] = None if state is None else normal(g, (n, D, E), state)
    i["df"] = None if state is None else normal(g, (n, D, E), state)
    return i, n


def forward(i, cu, n, state, softplus=True, carry=True, **kw):
    x = i["x"]
    (B, T, D), E = x.shape, i["A"].shape[1]
    y, fin = blank(x.shape, x.dtype), blank((n, D, E), state or F)
    c = blank(kda.ssm_carry_shape(B, T, D, E)) if carry else None
    kda.ssm_fwd(x, i["dt"], i["A"], i["B"], i["C"], y, D=i["skip"], z=i["z"], dt_bias=i["bias"], softplus=softplus,
                initial_state=i["h0"], final_state=fin, cu_seqlens=cu, carry=c, **kw)
    return y, fin, c


def backward(i, cu, n, carry, softplus=True, **kw):
    x = i["x"]
    D, E = i["A"].shape
    o = {"dx": blank(x.shape, x.dtype), "ddt": blank(x.shape, x.dtype), "dA": blank((D, E)), "dB": blank(i["B"].shape, x.dtype),
         "dC": blank(i["B"].shape, x.dtype), "d_initial": blank((n, D, E))}
    if i["skip"] is not None:
        o["dskip"] = blank((D,))
    if i["z"] is not None:
        o["dz"] = blank(x.shape, x.dtype)
    if i["bias"] is not None:
        o["dbias"] = blank((D,))
    kda.ssm_bwd(x, i["dt"], i["A"], i["B"], i["C"], i["dy"], carry, o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], D=i["skip"],
                d_D=o.get("dskip"), z=i["z"], d_z=o.get("dz"), dt_bias=i["bias"], d_dt_bias=o.get("dbias"), softplus=softplus,
                initial_state=i["h0"], d_final=i["df"], d_initial=o["d_initial"], cu_seqlens=cu, **kw)
    return o


def plain(i, sp, softplus=True, grad=True):
    f = lambda t: None if t is None else t.reshape(-1, *t.shape[2:])  # noqa: E731
    return pl.ssm(f(i["x"]), f(i["dt"]), i["A"], f(i["B"]), f(i["C"]), sp, i["skip"], f(i["z"]), i["bias"], softplus, i["h0"],
                  f(i["dy"]) if grad else None, i["df"] if grad else None)


TOKENS = ("y", "dx", "ddt", "dB", "dC", "dz")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("B,T,D,E,G,bounds", SHAPES)
def test_forward_and_backward(B, T, D, E, G, bounds, dtype):
    k = T + D + E
    state = [None, F, BF][k % 3]
    softplus = k % 4 != 1
    say("ssm", B, T, D, E, G, bounds, dtype, state, softplus)
    i, n = make(B, T, D, E, G, bounds, dtype, state)
    if not softplus:
        i["dt"] = (i["dt"].float().abs() * 0.3).to(dtype)
        i["bias"] = None if D % 2 else i["bias"].abs() * 0.05
    if k % 5 == 0:
        i["z"] = None
    if k % 7 == 0:
        i["skip"] = None
    sp = spans_of(bounds, B, T)
    rows, cu = covered(sp, B * T), cu_of(bounds)
    want = plain(i, sp, softplus)
    j = {a: gpu(t) for a, t in i.items()}
    y, fin, carry = forward(j, cu, n, state, softplus)
    got = {"y": y, "final": fin, **backward(j, cu, n, carry, softplus)}
    assert set(got) == set(want)
    for name, t in got.items():
        t = t.cpu()
        if name in TOKENS:
            t = t.reshape(-1, *t.shape[2:])
            pl.near(name, t, want[name], rows)
            untouched(name, t, rows)
        else:
            pl.near(name, t, want[name])
    again = backward(j, cu, n, carry, softplus, workspace=torch.full((kda.ssm_workspace_size(B, T, D, E, G, len(bounds) - 1 if bounds
                     else 0, True),), 255, dtype=torch.uint8, device=dev()))
    assert all(same(again[a], got[a]) for a in again)
    y2, fin2, _ = forward(j, cu, n, state, softplus, carry=False,
                          workspace=torch.full((kda.ssm_workspace_size(B, T, D, E, G, len(bounds) - 1 if bounds else 0),), 255,
                                               dtype=torch.uint8, device=dev()))
    assert same(y, y2) and same(fin, fin2)


def test_final_state_over_the_initial_one():
    """Sequences within a chunk, over chunks, and empty."""
    bounds = [0, 3, 130, 130, 131, 500, 520, 700]
    i, n = make(1, 700, 70, 16, 1, bounds, BF, F, 2)
    j, cu = {a: gpu(t) for a, t in i.items()}, cu_of(bounds)
    y, fin, _ = forward(j, cu, n, F)
    st, y2 = j["h0"].clone(), blank(y.shape, BF)
    kda.ssm_fwd(j["x"], j["dt"], j["A"], j["B"], j["C"], y2, D=j["skip"], z=j["z"], dt_bias=j["bias"], initial_state=st, final_state=st,
                cu_seqlens=cu)
    assert same(y, y2) and same(fin, st)
    # a sequence in pieces, each from the state that the one before has left
    j = {a: None if t is None else t[:1] if a == "h0" else t for a, t in j.items()}
    y, fin, _ = forward(j, None, 1, F)
    st, at = j["h0"].clone(), 0
    for hi in (64, 65, 300, 300, 700):
        p = {a: (t[:, at:hi].clone() if a in ("x", "dt", "B", "C", "z") else t) for a, t in j.items()}
        out = blank(p["x"].shape, BF)
        kda.ssm_fwd(p["x"], p["dt"], p["A"], p["B"], p["C"], out, D=p["skip"], z=p["z"], dt_bias=p["bias"], initial_state=st, final_state=st)
        # the same up to the rounding of where chunks are cut: bf16 outputs are a step apart at most
        d = (out.float() - y[:, at:hi].float()).abs()
        assert bool((d <= 2.0 ** -7 * y[:, at:hi].float().abs() + 1e-4).all())
        at = hi
    torch.testing.assert_close(st, fin, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("N,D,E,G", [(1, 1, 1, 1), (3, 129, 16, 1), (5, 66, 5, 3), (40, 520, 16, 2), (7, 30, 64, 1), (0, 8, 4, 1)])
@pytest.mark.parametrize("state", [F, BF], ids=str)
def test_step(N, D, E, G, dtype, state):
    say("ssm step", N, D, E, G, dtype, state)
    i, _ = make(1, N, D, E, G, None, dtype, None, N)
    g = torch.Generator().manual_seed(N)
    S = 2 * N + 3
    pool = normal(g, (S, D, E), state)
    perm = torch.randperm(S, generator=g).tolist()
    src, dst = perm[:N], perm[N:2 * N]
    if N >= 5:
        src[0], src[1], dst[2], dst[3] = -1, S, S + 5, src[3]
    j = {a: gpu(t[0]) if a in ("x", "dt", "B", "C", "z") else gpu(t) for a, t in i.items() if t is not None}
    p, y = gpu(pool), blank((N, D), dtype)
    kda.ssm_step(j["x"], j["dt"], j["A"], j["B"], j["C"], y, p, ints(src), ints(dst), D=j["skip"], z=j["z"], dt_bias=j["bias"])
    if N == 0:
        return
    i["h0"] = torch.stack([pool[s] if 0 <= s < S else torch.zeros(D, E, dtype=state) for s in src])
    i["df"] = None
    o = plain(i, [(k, k + 1) for k in range(N)], grad=False)
    pl.near("y", y.cpu(), o["y"])
    left = {d: k for k, d in enumerate(dst) if 0 <= d < S}
    for s in range(S):
        if s in left:
            pl.near("state", p[s].cpu(), o["final"][left[s]])
        else:
            assert torch.equal(p[s].cpu(), pool[s])


def test_nan_stays_in_its_sequence():
    bounds = [0, 70, 140, 210]
    i, n = make(1, 210, 40, 16, 1, bounds, F, F, 4)
    cu = cu_of(bounds)
    j = {a: gpu(t) for a, t in i.items()}
    bad = {a: None if t is None else t.clone() for a, t in j.items()}
    bad["x"][0, 100], bad["h0"][1, 3], bad["dy"][0, 139, 2], bad["df"][1, 5] = float("nan"), float("inf"), float("nan"), float("-inf")
    out = []
    for v in (j, bad):
        y, fin, carry = forward(v, cu, n, F)
        out.append({"y": y, "final": fin, **backward(v, cu, n, carry)})
    for k in TOKENS:
        a, b = out[0][k][0], out[1][k][0]
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[140:], b[140:]), k
    for k in ("final", "d_initial"):
        assert torch.equal(out[0][k][::2], out[1][k][::2]), k
    assert bool(torch.isnan(out[1]["y"][0, 100:140]).all())


@pytest.mark.parametrize("bias", [-60.0, -12.0, 0.0, 30.0, 100.0])
def test_far_steps(bias):
    """Softplus far from zero; decays of 1 and of 0."""
    i, n = make(1, 100, 24, 16, 1, None, F, F, 6)
    i["bias"] = torch.full((24,), bias)
    sp = [(0, 100)]
    want = plain(i, sp)
    j = {a: gpu(t) for a, t in i.items()}
    y, fin, carry = forward(j, None, 1, F)
    got = {"y": y, "final": fin, **backward(j, None, 1, carry)}
    for name, t in got.items():
        t = t.cpu()
        pl.near(name, t.reshape(-1, *t.shape[2:]) if name in TOKENS else t, want[name])


def test_captured_and_on_another_stream():
    bounds = [0, 90, 90, 400]
    i, n = make(1, 400, 48, 16, 2, bounds, BF, F, 7)
    j, cu = {a: gpu(t) for a, t in i.items()}, cu_of(bounds)
    wf = torch.empty(kda.ssm_workspace_size(1, 400, 48, 16, 2, n), dtype=torch.uint8, device=dev())
    wb = torch.empty(kda.ssm_workspace_size(1, 400, 48, 16, 2, n, True), dtype=torch.uint8, device=dev())

    def step():
        y, fin, carry = forward(j, cu, n, F, workspace=wf)
        return [y, fin, *backward(j, cu, n, carry, workspace=wb).values()]
    want = step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = step()
    st.synchronize()
    assert all(same(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        j["x"].mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        assert all(same(a, b) for a, b in zip(got, step())), k


def test_gradients_that_are_not_wanted():
    i, n = make(1, 100, 40, 16, 1, None, BF, F, 9)
    j = {a: gpu(t) for a, t in i.items()}
    carry = forward(j, None, 1, F)[2]
    want = backward(j, None, 1, carry)
    x = j["x"]
    dx, ddt, dA, dB, dC = (blank(t.shape, t.dtype) for t in (x, x, j["A"], j["B"], j["B"]))
    kda.ssm_bwd(x, j["dt"], j["A"], j["B"], j["C"], j["dy"], carry, dx, ddt, dA, dB, dC, D=j["skip"], z=j["z"], dt_bias=j["bias"],
                initial_state=j["h0"], d_final=j["df"])
    for a, b in zip((dx, ddt, dA, dB, dC), ("dx", "ddt", "dA", "dB", "dC")):
        assert same(a, want[b]), b


def test_values_behind_a_sequence_are_not_used():
    """NaN in tokens that no sequence covers, and in a state beside them."""
    bounds = [70, 75, 200]
    i, n = make(1, 330, 40, 16, 1, bounds, F, F, 10)
    cu = cu_of(bounds)
    j = {a: gpu(t) for a, t in i.items()}
    bad = {a: None if t is None else t.clone() for a, t in j.items()}
    for k in ("x", "dt", "B", "C", "z", "dy"):
        bad[k][:, :70], bad[k][:, 200:] = float("nan"), float("inf")
    out = []
    for v in (j, bad):
        y, fin, carry = forward(v, cu, n, F)
        out.append({"y": y, "final": fin, **backward(v, cu, n, carry)})
    for k in out[0]:
        assert same(out[0][k], out[1][k]), k
    # the last token's state alone is infinite: no sum over tokens uses it
    j["x"][0, 199] = float("inf")
    y, fin, carry = forward(j, cu, n, F)
    j["df"] = None
    j["dy"][0, 199] = 0
    got = backward({**j, "z": None, "skip": None}, cu, n, carry)
    assert bool(torch.isfinite(got["dA"]).all())


def test_two_calls_at_once():
    """Two streams, each with its own workspace."""
    i, n = make(1, 1500, 64, 16, 1, None, BF, None, 8)
    j = {a: gpu(t) for a, t in i.items()}
    want = forward(j, None, 1, None)[0]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([forward(j, None, 1, None)[0] for _ in range(4)])
    torch.cuda.synchronize()
    assert all(same(want, o) for s in outs for o in s)


def test_refusals():
    i, n = make(1, 8, 8, 4, 1, None, F, None)
    j = {a: gpu(t) for a, t in i.items()}
    y = blank(j["x"].shape)
    base = dict(x=j["x"], dt=j["dt"], A=j["A"], B=j["B"], C=j["C"], y=y)
    for bad in (dict(dt=j["dt"].to(BF)), dict(A=j["A"][:4]), dict(B=j["B"][..., :2]), dict(C=j["C"][0]), dict(D=j["skip"][:3]),
                dict(z=j["z"].to(BF)), dict(dt_bias=j["bias"].to(BF)), dict(carry=blank((2, 8, 4))), dict(initial_state=blank((1, 8, 3))),
                dict(initial_state=blank((1, 8, 4)), final_state=blank((1, 8, 4), BF)), dict(cu_seqlens=cu_of([0]))):
        with pytest.raises(ValueError):
            kda.ssm_fwd(**{**base, **bad})
    with pytest.raises(kda.KDAError):
        kda.ssm_fwd(**{**base, "y": j["x"]})
    with pytest.raises(ValueError):
        kda.ssm_bwd(j["x"], j["dt"], j["A"], j["B"], j["C"], j["dy"], blank((1, 8, 4)), y, blank(y.shape), blank((8, 4)),
                    blank(j["B"].shape), blank(j["B"].shape), d_D=blank((8,)))


def grows(D=24, E=4, T=700, seed=12):
    """Without softplus, s > 0: decays of channels with A > 0 grow by up to 1.8 a token, exp(115) over 64."""
    i, n = make(1, T, D, E, 1, None, F, F, seed)
    i["dt"] = i["dt"].abs() * 0.3 + 1.2
    i["bias"], i["z"] = None, None
    i["A"][::2] = -i["A"][::2] * 0.3
    i["A"].clamp_(max=1.2)
    i["h0"].zero_()
    i["df"] = None
    return i, n


def both(i, n, grad=True):
    j = {a: gpu(t) for a, t in i.items()}
    y, fin, carry = forward(j, None, n, F, softplus=False)
    return {"y": y, "final": fin, **(backward(j, None, n, carry, softplus=False) if grad else {})}


def compare(got, want):
    for name, t in got.items():
        t = t.cpu()
        assert bool(torch.isfinite(t).all()), name
        pl.near(name, t.reshape(-1, *t.shape[2:]) if name in TOKENS else t, want[name])


def test_growing_decays_of_states_that_are_zero():
    """Padding with zeros in front: the state stays 0, whatever a chunk's decay is."""
    T, first = 700, 660
    i, n = grows()
    i["x"][:, :first] = 0
    got = both(i, n, grad=False)   # (a gradient would pass fp32 on its way to the first token)
    assert bool((got["y"][:, :first] == 0).all())
    got["y"] = got["y"][:, first:]
    end = {a: t[:, first:] if a in ("x", "dt", "B", "C", "dy") else t for a, t in i.items()}
    compare(got, plain(end, [(0, T - first)], softplus=False, grad=False))


def test_growing_decays_of_gradients_that_are_zero():
    """No gradient from the last tokens: it stays 0 towards the first ones."""
    T, last = 700, 40
    i, n = grows(seed=13)
    i["x"].zero_()                 # (so that the states are 0)
    i["dy"][:, last:] = 0
    got = both(i, n)
    for name in TOKENS:
        if name in got:
            assert bool((got[name][:, last:] == 0).all()), name
            got[name] = got[name][:, :last]
    begin = {a: t[:, :last] if a in ("x", "dt", "B", "C", "dy") else t for a, t in i.items()}
    compare(got, plain(begin, [(0, last)], softplus=False))


@pytest.mark.parametrize("T", [192, 1344])
def test_growing_decays_of_states_that_are_small(T):
    """A chunk's decay of exp(95) times a state, or a gradient, far below 1: the products are in range."""
    i, n = grows(T=T, seed=14)
    g = torch.Generator().manual_seed(3)
    i["h0"], i["df"] = normal(g, i["h0"].shape), normal(g, i["h0"].shape)
    i["A"][::2], i["A"][1::2] = 1.2, -0.1
    # three blocks of 64 tokens with decays of about exp(-76), exp(95) and exp(-21)
    step = torch.tensor([-0.9, 1.13, -0.25])[torch.arange(T) // 64 % 3]
    i["dt"] = step[None, :, None] * (1.0 + 0.2 * torch.rand(i["dt"].shape, generator=g))
    i["x"][0, 5:] = 0
    i["dy"][0, :T - 5] = 0
    compare(both(i, n), plain(i, [(0, T)], softplus=False))


# chunks of several 64-token blocks in both directions: long packed batches, and wide ones (of narrow
# groups), where each workgroup's share of the channels is small
LONG = [(1, 17000, 16, 4, 1, None), (1, 17000, 16, 4, 1, [0, 5, 4000, 4000, 9000, 9001, 16999]), (2, 384, 1024, 4, 1024, None),
        (1, 800, 1024, 3, 1024, [3, 70, 333, 700]), (1, 4200, 256, 4, 128, [0, 1500, 1500, 4111]), (1, 2100, 520, 9, 260, None)]


@pytest.mark.parametrize("dtype", [BF, F], ids=str)
@pytest.mark.parametrize("B,T,D,E,G,bounds", LONG)
def test_chunks_of_several_blocks(B, T, D, E, G, bounds, dtype):
    say("ssm long", B, T, D, E, G, bounds, dtype)
    i, n = make(B, T, D, E, G, bounds, dtype, F, 15)
    i["A"][:, ::2] *= 0.01   # states that last over many chunks beside those that do not
    sp = spans_of(bounds, B, T)
    rows, cu = covered(sp, B * T), cu_of(bounds)
    want = plain(i, sp)
    j = {a: gpu(t) for a, t in i.items()}
    y, fin, carry = forward(j, cu, n, F)
    got = {"y": y, "final": fin, **backward(j, cu, n, carry)}
    assert set(got) == set(want)
    for name, t in got.items():
        t = t.cpu()
        if name in TOKENS:
            t = t.reshape(-1, *t.shape[2:])
            pl.near(name, t, want[name], rows)
            untouched(name, t, rows)
        else:
            pl.near(name, t, want[name])
    st, y2 = j["h0"].clone(), blank(y.shape, dtype)   # the final states over the initial ones
    kda.ssm_fwd(j["x"], j["dt"], j["A"], j["B"], j["C"], y2, D=j["skip"], z=j["z"], dt_bias=j["bias"], initial_state=st, final_state=st,
                cu_seqlens=cu)
    assert same(y, y2) and same(fin, st)


@pytest.mark.parametrize("B,T,D,E,G,bounds", LONG)
def test_sums_over_chunks_of_several_blocks(B, T, D, E, G, bounds):
    """d_D is the sum of dy x (without z): of whole numbers it is exact, and every token counts once."""
    i, n = make(B, T, D, E, G, bounds, F, None, 16)
    g = torch.Generator().manual_seed(17)
    i["x"], i["dy"] = (torch.randint(-3, 4, (B, T, D), generator=g).float() for _ in range(2))
    i["z"] = None
    rows, cu = covered(spans_of(bounds, B, T), B * T), cu_of(bounds)
    j = {a: gpu(t) for a, t in i.items()}
    carry = forward(j, cu, n, None)[2]
    got = backward(j, cu, n, carry)["dskip"].cpu()
    assert torch.equal(got.double(), (i["x"] * i["dy"]).double().reshape(-1, D)[rows].sum(0))
