"""The root-mean-square norm on the GPU against its plain 64-bit form."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_layer as pl
from gpu_util import BF, DTYPES, F, H16, blank, dev, gpu, normal, same, say

pytestmark = pytest.mark.gpu

E8 = torch.float8_e4m3fn
WIDTHS = [1, 7, 8, 127, 128, 129, 200, 512, 777, 1024, 2000, 2050, 4096, 5001, 8192, 9000, 16384, 16387, 20000]


def make(M, D, dtype, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return {"x": normal(g, (M, D), dtype, std), "res": normal(g, (M, D), dtype, 2 * std), "w": normal(g, (D,), std=0.3, mean=1.0),
            "dy": normal(g, (M, D), dtype), "dr": normal(g, (M, D), dtype)}


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", WIDTHS)
def test_forward_and_backward(D, dtype):
    M = 37 if D < 600 else 5
    i = make(M, D, dtype, D)
    eps = 1e-6
    for residual, weight in ((True, True), (False, False)):
        say("rmsnorm", M, D, dtype, residual, weight)
        res, w = (i["res"] if residual else None), (i["w"] if weight else None)
        s, r, y = pl.rmsnorm(i["x"], res, w, eps)
        x, got, ro, rstd = gpu(i["x"]), blank((M, D), dtype), blank((M, D), dtype), blank((M,))
        kda.rmsnorm_fwd(x, gpu(w), eps, got, residual=gpu(res), residual_out=ro, rstd=rstd)
        pl.near("y", got.cpu(), y)
        pl.near("rstd", rstd.cpu(), r)
        pl.near("residual_out", ro.cpu(), s)
        alone = blank((M, D), dtype)
        kda.rmsnorm_fwd(x, gpu(w), eps, alone, residual=gpu(res))
        assert same(alone, got)
        dr = i["dr"] if residual else None
        ro_c, rstd_c = ro.cpu(), rstd.cpu()
        dx_w, dw_w = pl.rmsnorm_bwd(i["dy"], ro_c, w, rstd_c, dr)
        dx, dw = blank((M, D), dtype), blank((D,))
        kda.rmsnorm_bwd(gpu(i["dy"]), ro, gpu(w), rstd, dx, d_weight=dw, d_residual=gpu(dr))
        pl.near("dx", dx.cpu(), dx_w)
        pl.near("dw", dw.cpu(), dw_w)
        a, b = blank((M, D), dtype), blank((D,))
        kda.rmsnorm_bwd(gpu(i["dy"]), ro, gpu(w), rstd, a, d_residual=gpu(dr))
        kda.rmsnorm_bwd(gpu(i["dy"]), ro, gpu(w), rstd, None, d_weight=b)
        assert same(a, dx) and same(b, dw)


def check_8bit(y8, scales, y, group):
    """Scales are the largest size / 448 within the bounds of y and one rounding of the quotient; a
    value is rounded to half a step of 3 mantissa bits (2^-4 of it; half of 2^-9 below 2^-6) from y
    over the scale that was given, which carries y's bound and three roundings."""
    M, D = y.v.shape
    for k in range(scales.shape[1]):
        c = slice(k * group, min(D, (k + 1) * group))
        v, e = y.v[:, c], y.e[:, c]
        top = v.abs().amax(1)
        sc = scales[:, k].double()
        want = top / 448
        slack = e.amax(1) / 448 + 2 * pl.U * want + 2.0 ** -149
        zero = top <= e.amax(1)
        assert bool((((sc - want).abs() <= slack) | (zero & (sc == 1))).all()), k
        q = v / sc[:, None]
        tol = e / sc[:, None] + 6 * pl.U * q.abs()
        got = y8[:, c].double()
        tol = tol + torch.maximum((q.abs() + tol) * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
        assert bool(torch.isfinite(got).all()) and bool(((got - q).abs() <= tol).all()), k


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", WIDTHS)
def test_8_bits(D, dtype):
    M = 19 if D < 600 else 3
    i = make(M, D, dtype, D + 1)
    i["x"][M // 2] = 0
    i["res"][M // 2] = 0
    if D > 200:
        i["x"][0, 130:200], i["res"][0, 130:200] = 0, 0
    s, r, y = pl.rmsnorm(i["x"], i["res"], i["w"], 1e-6)
    for group in sorted({128, D}):
        say("rmsnorm 8 bits", M, D, dtype, group)
        y8, ro, rstd = torch.full((M, D), 100.0, device=dev()).to(E8), blank((M, D), dtype), blank((M,))
        scales = blank((M, -(-D // group)))
        kda.rmsnorm_fwd(gpu(i["x"]), gpu(i["w"]), 1e-6, y8, residual=gpu(i["res"]), residual_out=ro, scales=scales, rstd=rstd)
        check_8bit(y8.float().cpu(), scales.cpu(), y, group)
        pl.near("residual_out", ro.cpu(), s)
        pl.near("rstd", rstd.cpu(), r)


@pytest.mark.parametrize("D", [64, 300, 20000])
@pytest.mark.parametrize("per_row", [True, False])
def test_8_bits_of_tiny_and_other_values(D, per_row):
    """Scales of which the reciprocal overflows, and values that are none."""
    i = make(6, D, F, 3)
    w = i["w"].clone()
    for row, size in enumerate((1e-38, 1e-43, 1e-30, 1e30)):
        say("tiny", D, size)
        wt = (torch.ones(D) * size)
        _, _, y = pl.rmsnorm(i["x"], None, wt, 0.0)
        scales = blank((6, 1 if per_row else -(-D // 128)))
        y8 = torch.empty(6, D, device=dev(), dtype=E8)
        kda.rmsnorm_fwd(gpu(i["x"]), gpu(wt), 0.0, y8, scales=scales)
        if size >= 1e-38:
            y.e.clamp_(min=2.0 ** -149)
            check_8bit(y8.float().cpu(), scales.cpu(), y, D if per_row else 128)
        assert bool(torch.isfinite(y8.float()).all()) and bool((scales > 0).all())
    x = i["x"].clone()
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y8, scales = torch.empty(6, D, device=dev(), dtype=E8), blank((6, 1 if per_row else -(-D // 128)))
    kda.rmsnorm_fwd(gpu(x), gpu(w), 1e-6, y8, scales=scales)
    sc = scales.cpu()
    assert bool(torch.isnan(sc[1]).all())        # the row's norm is NaN
    assert bool(torch.isnan(sc[2, 0]))           # infinity times 1 / infinity
    clean = blank((6, D))
    kda.rmsnorm_fwd(gpu(x), gpu(w), 1e-6, clean)
    assert bool(torch.isfinite(sc[[0, 3, 4, 5]]).all()) and bool(torch.isfinite(y8.float()[[0, 3, 4, 5]]).all())
    assert bool(torch.isfinite(clean[[0, 3, 4, 5]]).all()) and bool(torch.isnan(clean[1]).all())
    w[3] = float("inf")                           # one infinite value: the others are 0 beside it
    kda.rmsnorm_fwd(gpu(i["x"]), gpu(w), 1e-6, y8, scales=scales)
    assert bool(torch.isinf(scales[:, 0]).all()) and bool((y8.float()[:, :3] == 0).all()) and bool(torch.isnan(y8.float()[:, 3]).all())


@pytest.mark.parametrize("D", [96, 1500, 17000])
def test_in_place(D):
    i = make(9, D, BF, 5)
    w = gpu(i["w"])
    y, ro, rstd = blank((9, D), BF), blank((9, D), BF), blank((9,))
    kda.rmsnorm_fwd(gpu(i["x"]), w, 1e-6, y, residual=gpu(i["res"]), residual_out=ro, rstd=rstd)
    for swap in (False, True):
        x, res = gpu(i["x"]), gpu(i["res"])
        a, b = (res, x) if swap else (x, res)
        kda.rmsnorm_fwd(x, w, 1e-6, a, residual=res, residual_out=b)
        assert same(a, y) and same(b, ro)
    dx, dw = blank((9, D), BF), blank((D,))
    kda.rmsnorm_bwd(gpu(i["dy"]), ro, w, rstd, dx, d_weight=dw, d_residual=gpu(i["dr"]))
    for k in range(3):
        t = [gpu(i["dy"]), ro.clone(), gpu(i["dr"])]
        got = blank((D,))
        kda.rmsnorm_bwd(t[0], t[1], w, rstd, t[k], d_weight=got, d_residual=t[2])
        assert same(t[k], dx) and same(got, dw), k


def test_many_rows_empty_calls_and_graphs():
    """More rows than workgroups at once; no rows; captured."""
    i = make(70001, 16, H16, 6)
    s, r, y = pl.rmsnorm(i["x"], i["res"], i["w"], 1e-6)
    got, ro, rstd = blank((70001, 16), H16), blank((70001, 16), H16), blank((70001,))
    kda.rmsnorm_fwd(gpu(i["x"]), gpu(i["w"]), 1e-6, got, residual=gpu(i["res"]), residual_out=ro, rstd=rstd)
    pl.near("y", got.cpu(), y)
    dxw, dww = pl.rmsnorm_bwd(i["dy"], ro.cpu(), i["w"], rstd.cpu(), None)
    dx, dw = blank((70001, 16), H16), blank((16,))
    kda.rmsnorm_bwd(gpu(i["dy"]), ro, gpu(i["w"]), rstd, dx, d_weight=dw)
    pl.near("dx", dx.cpu(), dxw)
    pl.near("dw", dw.cpu(), dww)
    e = torch.empty(0, 40, device=dev())
    dw = blank((40,))
    kda.rmsnorm_fwd(e, None, 1e-6, e.clone())
    kda.rmsnorm_bwd(e, e, None, torch.empty(0, device=dev()), e.clone(), d_weight=dw)
    assert bool((dw == 0).all())
    i = make(300, 1000, BF, 7)
    x, res, w, dy = gpu(i["x"]), gpu(i["res"]), gpu(i["w"]), gpu(i["dy"])
    y, ro, rstd, dx, dw = blank(x.shape, BF), blank(x.shape, BF), blank((300,)), blank(x.shape, BF), blank((1000,))
    ws = torch.empty(kda.rmsnorm_workspace_size(300, 1000), dtype=torch.uint8, device=dev())

    def step():
        kda.rmsnorm_fwd(x, w, 1e-6, y, residual=res, residual_out=ro, rstd=rstd)
        kda.rmsnorm_bwd(dy, ro, w, rstd, dx, d_weight=dw, workspace=ws)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, ro, rstd, dx, dw)]
        step()
        assert all(same(a, b) for a, b in zip(got, (y, ro, rstd, dx, dw))), k


def test_refusals():
    x = torch.zeros(4, 256, device=dev())
    y8 = torch.empty(4, 256, device=dev(), dtype=E8)
    sc = torch.empty(4, 2, device=dev())
    for kw in (dict(y=y8), dict(y=y8, scales=torch.empty(4, 3, device=dev())), dict(y=y8, scales=torch.empty(8, device=dev())),
               dict(y=x.clone(), scales=sc), dict(y=x.to(BF)), dict(y=x.clone(), residual=x.to(BF)), dict(y=y8, scales=sc.to(H16)),
               dict(y=x.clone(), rstd=torch.empty(3, device=dev()))):
        with pytest.raises(ValueError):
            kda.rmsnorm_fwd(x, None, 1e-6, **kw)
    y = x.clone()
    with pytest.raises(kda.KDAError):
        kda.rmsnorm_fwd(x, None, 1e-6, y, residual_out=y)
    with pytest.raises(kda.KDAError):
        kda.rmsnorm_fwd(x, None, -1.0, y)
    with pytest.raises(ValueError):
        kda.rmsnorm_bwd(x, x, None, None, y)


@pytest.mark.parametrize("D", [64, 300, 2100, 20000])
@pytest.mark.parametrize("per_row", [True, False])
def test_8_bits_of_coarse_scales(D, per_row):
    """Scales of a few steps of 2^-149: the quotient can pass 448 by up to half, and is held there."""
    i = make(4, D, F, 8)
    group = D if per_row else 128
    for steps in (130, 180, 250, 400, 900, 2000):
        wt = torch.full((D,), steps * 2.0 ** -149)
        _, _, y = pl.rmsnorm(i["x"], None, wt, 0.0)
        scales, y8 = blank((4, -(-D // group))), torch.empty(4, D, device=dev(), dtype=E8)
        kda.rmsnorm_fwd(gpu(i["x"]), gpu(wt), 0.0, y8, scales=scales)
        got, sc = y8.float().cpu().double(), scales.cpu().double()
        for k in range(sc.shape[1]):
            c = slice(k * group, min(D, (k + 1) * group))
            v, s = y.v[:, c], sc[:, k, None]
            # y is rounded to whole steps, its largest / 448 to a whole one too
            assert bool(((s[:, 0] - v.abs().amax(1) / 448).abs() <= 2.0 ** -149).all()), (steps, k)
            q = (v / s).clamp(-448, 448)
            tol = 2.0 ** -149 / s + 1e-5 * q.abs()
            tol = tol + torch.maximum((q.abs() + tol) * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
            assert bool(((got[:, c] - q).abs() <= tol).all()), (steps, k)
            # t steps, t > 1/2, are rounded to 2 t at most: the largest quotient is not below 224
            assert bool((got[:, c].abs().amax(1) >= 224).all()), (steps, k)
