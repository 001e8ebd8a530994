"""The short causal convolution on the GPU against its plain 64-bit form."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_layer as pl
from gpu_util import BF, DTYPES, F, H16, blank, covered, cu_of, dev, gpu, ints, normal, same, say, spans_of, untouched

pytestmark = pytest.mark.gpu

RAGGED = [0, 1, 1, 3, 40, 41, 107, 107, 150]
# B, T, D, bounds of packed sequences
SHAPES = [(1, 1, 1, None), (2, 3, 5, None), (3, 17, 8, None), (2, 70, 67, None), (1, 150, 512, RAGGED), (1, 150, 130, RAGGED),
          (1, 150, 12, [7, 30, 30, 31, 140]), (1, 40, 3, [0, 40]), (4, 0, 16, None), (1, 0, 24, [0, 0, 0]), (1, 300, 4100, None)]


def make(B, T, D, W, bounds, dtype, state, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = len(bounds) - 1 if bounds else B
    i = {"x": normal(g, (B, T, D), dtype), "w": normal(g, (D, W), std=0.5), "b": normal(g, (D,), std=0.2),
         "dy": normal(g, (B, T, D), dtype)}
    i["h0"] = None if state is None else normal(g, (n, W - 1, D), state)
    i["df"] = None if state is None else normal(g, (n, W - 1, D), state)
    return i, n


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,D,bounds", SHAPES)
def test_forward_and_backward(B, T, D, bounds, W, dtype):
    state = [None, F, BF][(T + W) % 3]
    silu, bias = (D + W) % 4 != 0, D % 3 != 1
    say("conv", B, T, D, bounds, W, dtype, state, silu, bias)
    i, n = make(B, T, D, W, bounds, dtype, state)
    if not bias:
        i["b"] = None
    sp = spans_of(bounds, B, T)
    o = pl.conv(i["x"].reshape(-1, D), i["w"], i["b"], sp, i["h0"], silu, i["dy"].reshape(-1, D), i["df"])
    rows = covered(sp, B * T)
    x, w, b, dy, cu = gpu(i["x"]), gpu(i["w"]), gpu(i["b"]), gpu(i["dy"]), cu_of(bounds)
    y, fin = blank(x.shape, dtype), blank((n, W - 1, D), state or F)
    kda.conv_fwd(x, w, b, y, initial_state=gpu(i["h0"]), final_state=fin, cu_seqlens=cu, silu=silu)
    pl.near("y", y.cpu().reshape(-1, D), o["y"], rows)
    untouched("y", y.cpu().reshape(-1, D), rows)
    pl.near("final", fin.cpu(), o["final"])
    dx, dw, db = blank(x.shape, dtype), blank(w.shape), None if b is None else blank(b.shape)
    d0 = blank((n, W - 1, D))
    args = dict(d_weight=dw, d_bias=db, initial_state=gpu(i["h0"]), d_final=gpu(i["df"]), d_initial=d0, cu_seqlens=cu, silu=silu)
    kda.conv_bwd(x, w, b, dy, dx, **args)
    pl.near("dx", dx.cpu().reshape(-1, D), o["dx"], rows)
    untouched("dx", dx.cpu().reshape(-1, D), rows)
    pl.near("dw", dw.cpu(), o["dw"])
    if db is not None:
        pl.near("db", db.cpu(), o["db"])
    pl.near("d_initial", d0.cpu(), o["d_initial"])
    first = [t.clone() for t in (dx, dw, d0)]
    ws = torch.full((max(1, kda.conv_workspace_size(B, T, D, W)),), 255, dtype=torch.uint8, device=dev())
    kda.conv_bwd(x, w, b, dy, dx, **args, workspace=ws)   # the same bits, whatever the workspace held
    assert all(same(a, c) for a, c in zip(first, (dx, dw, d0)))
    kda.conv_bwd(x, w, b, dy, dx, initial_state=gpu(i["h0"]), d_final=gpu(i["df"]), cu_seqlens=cu, silu=silu)
    assert same(first[0], dx)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("N,D,W", [(1, 1, 2), (3, 129, 4), (5, 64, 3), (70, 520, 4), (0, 8, 4)])
@pytest.mark.parametrize("state", [F, BF], ids=str)
def test_step(N, D, W, dtype, state):
    say("conv step", N, D, W, dtype, state)
    g = torch.Generator().manual_seed(N)
    S = 2 * N + 3
    x, w, b, pool = normal(g, (N, D), dtype), normal(g, (D, W)), normal(g, (D,)), normal(g, (S, W - 1, D), state)
    perm = torch.randperm(S, generator=g).tolist()
    src, dst = perm[:N], perm[N:2 * N]
    if N >= 5:
        src[0], src[1], dst[2] = -1, S + 7, -1      # from zeros, and left nowhere
        dst[3] = src[3]                              # in place
        src[4] = perm[N + 6 if N > 6 else 0] if N > 6 else src[4]
        if N > 6:
            dst[6] = S                               # (its slot is read by sequence 4)
    h0 = torch.stack([pool[s] if 0 <= s < S else torch.zeros(W - 1, D, dtype=state) for s in src]) if N else torch.zeros(0, W - 1, D)
    o = pl.conv(x, w, b, [(k, k + 1) for k in range(N)], h0) if N else None
    p, y = gpu(pool), blank((N, D), dtype)
    kda.conv_step(gpu(x), gpu(w), gpu(b), y, p, ints(src), ints(dst))
    if N == 0:
        return
    pl.near("y", y.cpu(), o["y"])
    left = {d: k for k, d in enumerate(dst) if 0 <= d < S}
    for s in range(S):
        if s in left:
            pl.near("state", p[s].cpu(), o["final"][left[s]])
        else:
            assert torch.equal(p[s].cpu(), pool[s])


def test_chunks_of_a_sequence_in_place():
    """A sequence in pieces, its state over the one before, is the sequence at once."""
    i, _ = make(1, 130, 72, 4, None, BF, None, 3)
    x, w, b = gpu(i["x"]), gpu(i["w"]), gpu(i["b"])
    y, st = blank(x.shape, BF), torch.zeros(1, 3, 72, device=dev())
    kda.conv_fwd(x, w, b, y)
    for lo, hi in ((0, 1), (1, 3), (3, 64), (64, 64), (64, 130)):
        part = blank((1, hi - lo, 72), BF)
        kda.conv_fwd(x[:, lo:hi].contiguous(), w, b, part, initial_state=st, final_state=st)
        assert same(part, y[:, lo:hi])
    assert torch.equal(st[0], x[0, -3:].float())


def test_nan_stays_in_its_sequence():
    i, _ = make(1, 60, 16, 4, [0, 20, 40, 60], F, F, 4)
    cu = cu_of([0, 20, 40, 60])
    x, w, b, dy = gpu(i["x"]), gpu(i["w"]), gpu(i["b"]), gpu(i["dy"])
    bad = x.clone()
    bad[0, 25], bad[0, 39, 3] = float("nan"), float("inf")
    out = []
    for v in (x, bad):
        y, dx, fin, d0 = blank(x.shape), blank(x.shape), blank((3, 3, 16)), blank((3, 3, 16))
        kda.conv_fwd(v, w, b, y, initial_state=gpu(i["h0"]), final_state=fin, cu_seqlens=cu)
        kda.conv_bwd(v, w, b, dy, dx, initial_state=gpu(i["h0"]), d_final=gpu(i["df"]), d_initial=d0, cu_seqlens=cu)
        out.append((y, dx, fin, d0))
    for k in (0, 1):
        assert torch.equal(out[0][k][0, :20], out[1][k][0, :20]) and torch.equal(out[0][k][0, 40:], out[1][k][0, 40:])
    assert torch.equal(out[0][0][0, 20:25], out[1][0][0, 20:25]) and bool(torch.isnan(out[1][0][0, 25:29]).all())
    for k in (2, 3):
        assert torch.equal(out[0][k][::2], out[1][k][::2])


@pytest.mark.parametrize("value", [-3e38, -200.0, -90.0, 90.0, 3e38])
def test_far_values(value):
    """SiLU far from zero: no NaN from an exponential that overflows."""
    x = torch.full((1, 8, 8), value, device=dev())
    w = torch.zeros(8, 2, device=dev())
    w[:, 1] = 1
    y = blank(x.shape)
    kda.conv_fwd(x, w, None, y)
    o = pl.conv(x.cpu().reshape(8, 8), w.cpu(), None, [(0, 8)])
    pl.near("y", y.cpu().reshape(8, 8), o["y"])


def test_captured_and_on_another_stream():
    i, n = make(1, 150, 64, 4, RAGGED, H16, F, 5)
    x, w, b, dy, cu, h0, df = (gpu(i[k]) if k in i else cu_of(RAGGED) for k in ("x", "w", "b", "dy", "cu", "h0", "df"))
    y, fin, dx, dw, db, d0 = blank(x.shape, H16), blank(h0.shape), blank(x.shape, H16), blank(w.shape), blank(b.shape), blank(h0.shape)
    ws = torch.empty(kda.conv_workspace_size(1, 150, 64, 4), dtype=torch.uint8, device=dev())

    def step():
        kda.conv_fwd(x, w, b, y, initial_state=h0, final_state=fin, cu_seqlens=cu)
        kda.conv_bwd(x, w, b, dy, dx, d_weight=dw, d_bias=db, initial_state=h0, d_final=df, d_initial=d0, cu_seqlens=cu, workspace=ws)
    outs = (y, fin, dx, dw, db, d0)
    step()
    want = [t.clone() for t in outs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for t in outs:
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    assert all(same(a, c) for a, c in zip(want, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for t in outs:
            t.fill_(float("nan"))
        x.copy_(gpu(i["x"]) * (1 + k))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(same(a, c) for a, c in zip(got, outs)), k


def test_versions_and_refusals():
    x, w = torch.zeros(1, 4, 8, device=dev()), torch.zeros(8, 4, device=dev())
    y = torch.empty_like(x)
    v = y._version
    kda.conv_fwd(x, w, None, y)
    assert y._version > v
    for bad, err in ((dict(weight=w[:, :1].contiguous()), kda.KDAError), (dict(weight=w.to(BF)), ValueError), (dict(y=y[:, :2]), ValueError),
                     (dict(x=x.transpose(1, 2)), ValueError), (dict(bias=w[0]), ValueError), (dict(y=x), kda.KDAError)):
        a = dict(x=x, weight=w, bias=None, y=y)
        a.update(bad)
        with pytest.raises(err):
            kda.conv_fwd(**a)
    with pytest.raises(ValueError):
        kda.conv_fwd(x, w, None, y, initial_state=torch.zeros(1, 4, 8, device=dev()))
    with pytest.raises(ValueError):
        kda.conv_fwd(x, w, None, y, initial_state=torch.zeros(1, 3, 8, device=dev(), dtype=H16))


@pytest.mark.parametrize("state", [F, BF], ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [4, 12, 20, 33])
def test_states_that_begin_at_any_element(D, dtype, state):
    """Where rows are no whole vectors of the token tensors, states may begin at any element (as layers
    of a cache do): the same bits as from aligned ones."""
    D += dtype == F and D % 4 == 0
    say("conv states", D, dtype, state)
    bounds = [0, 2, 2, 19, 60]
    i, n = make(1, 60, D, 4, bounds, dtype, state, 3)
    j, cu = {a: gpu(t) for a, t in i.items()}, cu_of(bounds)

    def run(off):
        def at(t=None):   # a copy, or an output, `off` elements into its memory
            v = blank((n * 3 * D + 8,), state)[off:off + n * 3 * D].view(n, 3, D)
            return v if t is None else v.copy_(t)
        y, fin, d0, dx = blank(j["x"].shape, dtype), at(), at(), blank(j["x"].shape, dtype)
        h0, df = at(j["h0"]), at(j["df"])
        kda.conv_fwd(j["x"], j["w"], j["b"], y, initial_state=h0, final_state=fin, cu_seqlens=cu)
        kda.conv_bwd(j["x"], j["w"], j["b"], j["dy"], dx, initial_state=h0, d_final=df, d_initial=d0, cu_seqlens=cu)
        return y, fin, dx, d0
    want = run(0)
    assert not any(bool(torch.isnan(t).any()) for t in want)
    for off in (1, 2, 3):
        assert all(same(a, b) for a, b in zip(run(off), want)), off
