"""The plain 64-bit gradients that the GPU tests compare against, against differences (CPU)."""
import pytest
import torch

import plain_layer as pl

f64 = torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(value, inputs, grads, seed, h=1e-6):
    """A directional derivative of value(inputs) by a central difference, whose error is h^2 of the
    third derivative and 1e-16 / h of the value, against the gradients."""
    for name in grads:
        d = torch.randn(inputs[name].shape, generator=gen(seed), dtype=f64)
        up, down = dict(inputs), dict(inputs)
        up[name], down[name] = inputs[name] + h * d, inputs[name] - h * d
        want = (value(up) - value(down)) / (2 * h)
        got = (grads[name] * d).sum()
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), (name, float(got), float(want))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv(W, silu):
    g, sp, D = gen(W), [(0, 1), (1, 1), (1, 9), (10, 12)], 3
    r = lambda *s: torch.randn(*s, generator=g, dtype=f64)  # noqa: E731
    i = {"x": r(12, D), "w": r(D, W), "b": r(D), "h0": r(4, W - 1, D)}
    dy, df = r(12, D), r(4, W - 1, D)
    dy[9] = 0

    def value(j):
        o = pl.conv(j["x"], j["w"], j["b"], sp, j["h0"], silu)
        return (torch.nan_to_num(o["y"].v) * dy).sum() + (o["final"].v * df).sum()
    o = pl.conv(i["x"], i["w"], i["b"], sp, i["h0"], silu, dy, df)
    check(value, i, {"x": torch.nan_to_num(o["dx"].v), "w": o["dw"].v, "b": o["db"].v, "h0": o["d_initial"].v}, W)


@pytest.mark.parametrize("softplus,gated,groups", [(True, True, 1), (False, False, 2), (True, False, 4)])
def test_ssm(softplus, gated, groups):
    g, sp, T, D, E = gen(groups), [(0, 6), (6, 6), (6, 7), (7, 12)], 12, 4, 3
    r = lambda *s: torch.randn(*s, generator=g, dtype=f64)  # noqa: E731
    i = {"x": r(T, D), "dt": r(T, D), "A": -torch.rand(D, E, generator=g, dtype=f64), "B": r(T, groups, E), "C": r(T, groups, E),
         "skip": r(D), "z": r(T, D), "bias": r(D), "h0": r(4, D, E)}
    if not gated:
        i["z"] = None
    dy, df = r(T, D), r(4, D, E)

    def run(j, **k):
        return pl.ssm(j["x"], j["dt"], j["A"], j["B"], j["C"], sp, j["skip"], j["z"], j["bias"], softplus, j["h0"], **k)

    def value(j):
        o = run(j)
        return (o["y"].v * dy).sum() + (o["final"].v * df).sum()
    o = run(i, dy=dy, d_final=df)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "skip": "dskip", "bias": "dbias", "h0": "d_initial"}
    if gated:
        names["z"] = "dz"
    check(value, i, {k: o[n].v for k, n in names.items()}, 5)


@pytest.mark.parametrize("D", [1, 5, 40])
def test_rmsnorm(D):
    g = gen(D)
    i = {"x": torch.randn(6, D, generator=g, dtype=f64), "w": torch.randn(D, generator=g, dtype=f64)}
    dy, dr = torch.randn(6, D, generator=g, dtype=f64), torch.randn(6, D, generator=g, dtype=f64)

    def value(j):
        s, _, y = pl.rmsnorm(j["x"], None, j["w"], 1e-2)
        return (y.v * dy).sum() + (s.v * dr).sum()
    dx, dw = pl.rmsnorm_bwd(dy, i["x"], i["w"], pl.rmsnorm(i["x"], None, i["w"], 1e-2)[1].v, dr)
    check(value, i, {"x": dx.v, "w": dw.v}, 3)


def test_reorder_lists():
    pool = torch.arange(8.0).view(1, 8, 1)
    new, after = pl.reorder(pool, [[5, 1, 3, 0]], [[2, 2, 0, 2]])
    assert new == [[3, 1, 5, 0]] and after.view(-1).tolist() == [3, 3, 2, 3, 4, 5, 6, 7]
    new, after = pl.reorder(pool, [[5, 1, 9]], [[-1, 1, 1]])
    assert new == [[5, 1, 9]] and torch.equal(after, pool)


def test_beam_lists():
    x = torch.log(torch.tensor([[[0.5, 0.25, 0.25], [0.25, 0.5, 0.25]]]))
    t, p, s = pl.beam(x, torch.tensor([[0.0, 0.0]]), 4)
    assert t == [[0, 1, 1, 2]] and p == [[0, 1, 0, 0]]
    t, p, s = pl.beam(x, torch.tensor([[0.0, -0.125]]), 3, torch.tensor([[0, 1]]), eos=2)
    assert t == [[2, 0, 1]] and p == [[1, 0, 0]] and s[0][0] == -0.125
