"""Layer norm on the GPU against its 64-bit form, forward and backward: types, widths from one
element to rows longer than registers hold, few and many rows, rows of one value, outputs over
inputs, graphs and streams."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_ops as po

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def say(*a):
    print("[gpu-test]", *a, flush=True)


def inputs(M, D, dtype, seed=0, affine=True, offset=0.3):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, D, generator=gen) * 1.5 + offset).to(dtype)
    dy = torch.randn(M, D, generator=gen).to(dtype)
    w = torch.randn(D, generator=gen) * 0.3 + 1 if affine else None
    b = torch.randn(D, generator=gen) * 0.2 if affine else None
    return x, dy, w, b


def to_dev(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


def run(x, dy, w, b, eps=EPS):
    M, D = x.shape
    xg, dyg, wg, bg = to_dev(x, dy, w, b)
    nan = lambda *s: torch.full(s, float("nan"), device=dev())
    o = {"y": torch.full_like(xg, float("nan")), "mean": nan(M), "rstd": nan(M), "dx": torch.full_like(xg, float("nan")),
         "dw": nan(D), "db": nan(D)}
    kda.layernorm_fwd(xg, wg, bg, eps, o["y"], mean=o["mean"], rstd=o["rstd"])
    kda.layernorm_bwd(dyg, xg, wg, o["mean"], o["rstd"], o["dx"], d_weight=o["dw"], d_bias=o["db"])
    torch.cuda.synchronize()
    return o


def check(x, dy, w, b, o, eps=EPS):
    v, e = po.layernorm(x, w, b, eps)
    for k in v:
        po.assert_near(k, o[k], v[k], e[k])
    v, e = po.layernorm_bwd(dy, x, w, o["mean"].cpu(), o["rstd"].cpu())
    for k in v:
        po.assert_near(k, o[k], v[k], e[k])


@pytest.mark.parametrize("dtype", [BF, HF, F], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 64, 100, 127, 128, 136, 256, 513, 1000, 1024, 2048, 4104, 8192, 12288, 16384, 20001, 40960, 1027, 2051, 4001, 6007, 13001])
@pytest.mark.parametrize("M", [1, 5, 131])
def test_sizes(dtype, D, M):
    say("layer norm", dtype, M, D)
    a = inputs(M, D, dtype, seed=D + M)
    check(*a, run(*a))


@pytest.mark.parametrize("M,D", [(70001, 128), (30000, 64), (9000, 1000), (5000, 33), (3001, 2048)])
def test_many_rows(M, D):
    say("many rows", M, D)
    a = inputs(M, D, BF, seed=1)
    check(*a, run(*a))


def test_no_weight_no_bias():
    say("no weight, no bias, and one of them")
    x, dy, w, b = inputs(50, 300, BF, seed=2)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check(x, dy, ww, bb, run(x, dy, ww, bb))


def test_rows_of_one_value_and_far_from_zero():
    """A row of one value is its bias with rstd = eps^-1/2; a mean of 200 beside a deviation of
    1.5 costs what rounding x costs, not the square of it."""
    say("constant rows, large means")
    x, dy, w, b = inputs(40, 520, F, seed=3, offset=200.0)
    x[3] = 5.0
    x[7] = 0.0
    o = run(x, dy, w, b)
    v, e = po.layernorm(x, w, b, EPS)
    for k in v:
        po.assert_near(k, o[k], v[k], e[k])
    assert torch.equal(o["y"][3].cpu(), b) and torch.equal(o["y"][7].cpu(), b)
    assert abs(float(o["rstd"][3]) - EPS ** -0.5) <= 4 * po.U * EPS ** -0.5


def test_rows_with_nan_and_infinities_stay_alone():
    say("NaN and infinities in some rows")
    x, dy, w, b = inputs(64, 200, BF, seed=4)
    clean = run(x, dy, w, b)
    x[9, 3], x[20, 0], x[21, :] = float("nan"), float("inf"), float("-inf")
    o = run(x, dy, w, b)
    keep = [m for m in range(64) if m not in (9, 20, 21)]
    for k in ("y", "mean", "rstd", "dx"):
        assert torch.equal(o[k][keep], clean[k][keep]), k
    assert torch.isnan(o["y"][9]).all() and torch.isnan(o["y"][21]).all()


def test_outputs_over_inputs():
    say("y over x, dx over dy and over x")
    for M, D in ((33, 128), (9, 1001), (5, 8192), (3, 40000)):
        x, dy, w, b = inputs(M, D, BF, seed=5)
        ref = run(x, dy, w, b)
        xg, dyg, wg, bg = to_dev(x, dy, w, b)
        y = xg.clone()
        kda.layernorm_fwd(y, wg, bg, EPS, y)
        assert torch.equal(y, ref["y"])
        for over in (0, 1):
            t = [dyg.clone(), xg.clone()]
            dw, db = torch.empty(D, device=dev()), torch.empty(D, device=dev())
            kda.layernorm_bwd(t[0], t[1], wg, ref["mean"], ref["rstd"], t[over], d_weight=dw, d_bias=db)
            assert torch.equal(t[over], ref["dx"]) and torch.equal(dw, ref["dw"]) and torch.equal(db, ref["db"])


def test_some_outputs_only():
    say("dx alone, the parameters' gradients alone, one of them")
    x, dy, w, b = inputs(300, 264, BF, seed=6)
    ref = run(x, dy, w, b)
    xg, dyg, wg = to_dev(x, dy, w)
    dx, dw, db = torch.empty_like(xg), torch.empty(264, device=dev()), torch.empty(264, device=dev())
    kda.layernorm_bwd(dyg, xg, wg, ref["mean"], ref["rstd"], dx)
    assert torch.equal(dx, ref["dx"])
    kda.layernorm_bwd(dyg, xg, wg, ref["mean"], ref["rstd"], None, d_weight=dw)
    assert torch.equal(dw, ref["dw"])
    kda.layernorm_bwd(dyg, xg, wg, ref["mean"], ref["rstd"], None, d_bias=db)
    assert torch.equal(db, ref["db"])
    kda.layernorm_bwd(dyg, xg, wg, ref["mean"], ref["rstd"], None)


def test_no_rows():
    say("M = 0")
    e = torch.empty(0, 40, dtype=BF, device=dev())
    z = torch.empty(0, device=dev())
    dw, db = torch.full((40,), 9.0, device=dev()), torch.full((40,), 9.0, device=dev())
    kda.layernorm_fwd(e, None, None, EPS, e, mean=z, rstd=z)
    kda.layernorm_bwd(e, e, None, z, z, e, d_weight=dw, d_bias=db)
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0


def test_heads_of_a_read_out():
    """[B, T, H, 128] as kda_fwd writes it: a row per token and head."""
    say("rows of a 4-D tensor")
    x = torch.randn(2, 30, 5, 128, generator=torch.Generator().manual_seed(7)).to(BF)
    y = torch.empty_like(x, device=dev())
    mean = torch.empty(2, 30, 5, device=dev())
    kda.layernorm_fwd(x.to(dev()), None, None, EPS, y, mean=mean)
    v, e = po.layernorm(x.reshape(-1, 128), None, None, EPS)
    po.assert_near("y", y.reshape(-1, 128), v["y"], e["y"])
    po.assert_near("mean", mean.reshape(-1), v["mean"], e["mean"])


def test_gradients_against_differences():
    """Central differences of step 1e-5 of the 64-bit form: its third derivative is below a
    hundred of the absolute sum here, so 1e-10 * 100 / 6 and 1e-16 / 1e-5 are far below 1e-4."""
    say("gradients against differences")
    x, dy, w, b = inputs(6, 50, F, seed=8)
    o = run(x, dy, w, b)
    f = torch.float64
    gen = torch.Generator().manual_seed(1)
    p = {"x": x.to(f), "w": w.to(f), "b": b.to(f)}
    for name, grad in (("x", o["dx"]), ("w", o["dw"]), ("b", o["db"])):
        d = torch.randn(p[name].shape, generator=gen, dtype=f)

        def loss(step):
            q = dict(p)
            q[name] = p[name] + step * d
            v, _ = po.layernorm(q["x"], q["w"], q["b"], EPS)
            return (v["y"] * dy.to(f)).sum()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = grad.cpu().to(f) * d
        assert abs(terms.sum() - want) <= 1e-4 * terms.abs().sum(), name


def test_same_bits_again():
    say("the same call gives the same bits")
    a = inputs(20000, 128, BF, seed=9)
    r = run(*a)
    for _ in range(3):
        o = run(*a)
        assert all(torch.equal(o[k], r[k]) for k in r)


def test_offsets_past_32_bits():
    say("offsets past 2^31 elements")
    d = dev()
    M, D = (1 << 31) // 4096 + 40, 4096
    x = torch.randn(M, D, device=d, dtype=BF, generator=torch.Generator(device=d).manual_seed(0))
    w = torch.rand(D, device=d)
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device=d), torch.empty(M, device=d)
    kda.layernorm_fwd(x, w, None, EPS, y, mean=mean, rstd=rstd)
    ys = torch.empty(40, D, device=d, dtype=BF)
    kda.layernorm_fwd(x[-40:].contiguous(), w, None, EPS, ys)
    assert torch.equal(y[-40:], ys)
    dx, dxs = torch.empty_like(x), torch.empty_like(ys)
    dw, db = torch.empty(D, device=d), torch.empty(D, device=d)
    kda.layernorm_bwd(y, x, w, mean, rstd, dx, d_weight=dw, d_bias=db)
    kda.layernorm_bwd(ys, x[-40:].contiguous(), w, mean[-40:].contiguous(), rstd[-40:].contiguous(), dxs)
    assert torch.equal(dx[-40:], dxs)
    # y = xhat w rounded to bf16, summed over the rows in fp64 (a part at a time)
    want = sum(y[i:i + 65536].double().sum(0) for i in range(0, M, 65536))
    bound = (64 + M / 64 + 1024) * po.U * sum(y[i:i + 65536].double().abs().sum(0) for i in range(0, M, 65536))
    assert bool(((db.double() - want).abs() <= bound).all())


def test_graph_replays():
    say("graph of forward and backward")
    x, dy, w, b = inputs(3000, 128, BF, seed=10)
    xg, dyg, wg, bg = to_dev(x, dy, w, b)
    ws = torch.empty(kda.layernorm_workspace_size(3000, 128), dtype=torch.uint8, device=dev())

    def buffers():
        return {"y": torch.empty_like(xg), "mean": torch.empty(3000, device=dev()), "rstd": torch.empty(3000, device=dev()),
                "dx": torch.empty_like(xg), "dw": torch.empty(128, device=dev()), "db": torch.empty(128, device=dev())}

    def step(o):
        kda.layernorm_fwd(xg, wg, bg, EPS, o["y"], mean=o["mean"], rstd=o["rstd"])
        kda.layernorm_bwd(dyg, xg, wg, o["mean"], o["rstd"], o["dx"], d_weight=o["dw"], d_bias=o["db"], workspace=ws)

    o = buffers()
    step(o)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(o)
    for seed in (1, 2, 3):
        n = inputs(3000, 128, BF, seed=20 + seed)
        for t, v in zip((xg, dyg, wg, bg), n):
            t.copy_(v)
        gr.replay()
        e = buffers()
        step(e)
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], e[k]) for k in o), seed


@pytest.mark.parametrize("value,D,dtype", [(v, D, F) for v in (0.1, 12345.678, 1e6 + 0.37, -3e-5) for D in (96, 100, 1000, 8192, 20001)]
                         + [(201.0, 300001, BF)])
def test_rows_of_one_value_give_the_bias(value, D, dtype):
    """y of a row of one value is its bias to the bit, and the mean is that value, also where the
    sum of D of them is rounded. The first mean is off by at most 31 roundings (a lane adds up
    to 20 terms, ten levels of partial sums, the division; of the bf16 rows the 296 terms of a
    lane add up exactly, below 2^24 of the value's last places), so by less than 62 half units
    in the value's last place (22 for the bf16 rows). The differences from it are whole numbers
    of those: their sums, below 62 * 20001 and 22 * 300001 and so below 2^24 of them, are exact,
    so is their mean, and what is left of each difference is zero. rstd: the squares' mean and
    the mean's square differ by at most 31 u of them."""
    say("rows of", value, D, dtype)
    x = torch.full((3, D), value).to(dtype)
    _, dy, w, b = inputs(3, D, dtype, seed=11)
    o = run(x, dy, w, b)
    assert torch.equal(o["y"].cpu(), b.to(dtype).expand(3, D))
    assert torch.equal(o["mean"].cpu(), x[:, 0].float())
    off = 31 * po.U * abs(value)   # of the first mean
    worst = 31 * po.U * off ** 2 / EPS
    assert bool(((o["rstd"].cpu() / EPS ** -0.5 - 1).abs() <= worst + 8 * po.U).all())
    assert torch.isfinite(o["dx"]).all()


@pytest.mark.parametrize("D", [100, 1000, 8192, 20001])
@pytest.mark.parametrize("offset", [1e4, -3e5])
def test_rows_far_from_zero(offset, D):
    """fp32 rows of deviation 1.5 around 1e4 and -3e5. x - m is exact beside any m within a
    factor of two; a sum of D such terms takes at most 31 roundings (as above). So with xh the
    exact normalised values: centred values are off by u of themselves and 33 u of their mean
    absolute value, the variance by 36 u of itself and rstd by 22 u, and the products add 3:
    28 u of |xh| and 33 u of its mean, times the weight, and 2 u of y's two terms."""
    say("rows around", offset, D)
    x, dy, w, b = inputs(9, D, F, seed=12, offset=offset)
    o = run(x, dy, w, b)
    f = torch.float64
    c = x.to(f) - x.to(f).mean(1, keepdim=True)
    rstd = (c.square().mean(1, keepdim=True) + EPS) ** -0.5
    xh = c * rstd
    u = po.U
    bound = w.abs().to(f) * (28 * u * xh.abs() + 33 * u * xh.abs().mean(1, keepdim=True)) + 2 * u * ((xh * w).abs() + b.abs())
    po.assert_near("y", o["y"], xh * w.to(f) + b.to(f), bound)
    po.assert_near("mean", o["mean"], x.to(f).mean(1), 33 * u * c.abs().mean(1))
    po.assert_near("rstd", o["rstd"], rstd[:, 0], 22 * u * rstd[:, 0])
