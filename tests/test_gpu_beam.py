"""Beam search on the GPU: selection against sorting all continuations in 64 bits, and the beams'
states in a cache against plain lists."""
import pytest
import torch

import gated_delta_rule_87_amd as kda
import plain_layer as pl
from gpu_util import BF, DTYPES, F, H16, blank, dev, gpu, ints, normal, same, say

pytestmark = pytest.mark.gpu


def select(logits, scores, k, finished=None, eos=0, **kw):
    N, W, V = logits.shape
    t, p = torch.full((N, k), -99, dtype=torch.int32, device=dev()), torch.full((N, k), -99, dtype=torch.int32, device=dev())
    s = blank((N, k))
    kda.beam_select(logits, scores, t, p, s, finished=finished, eos=eos, **kw)
    return t, p, s


def check(logits, scores, k, finished=None, eos=0):
    """The same continuations in the same order, and scores to half a step of fp32 (64-bit sums are
    off by 1e-10 at most; finite ones that round to infinity are compared as such)."""
    want = pl.beam(logits, scores, k, finished, eos)
    t, p, s = select(gpu(logits), gpu(scores), k, gpu(finished), eos)
    assert t.tolist() == want[0] and p.tolist() == want[1]
    w = torch.tensor(want[2], dtype=torch.float64)
    got = s.cpu().double()
    ok = (got == w) | ((got - w).abs() <= 2.0 ** -24 * w.abs() + 1e-9)
    assert bool(ok.all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("N,W,V,k", [(1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 7, 4), (1, 4, 2048, 4), (3, 4, 2049, 8), (2, 5, 5003, 16),
                                     (1, 64, 100, 64), (2, 2, 20000, 64), (9, 8, 60000, 8), (1, 1, 100001, 33), (70, 4, 9001, 2),
                                     (54, 11, 586, 11), (1, 2, 2996, 2), (2, 3, 600, 64), (130, 4, 8200, 40)])
def test_select(N, W, V, k, dtype):
    say("beam", N, W, V, k, dtype)
    g = torch.Generator().manual_seed(V)
    logits, scores = normal(g, (N, W, V), dtype, 3.0), -torch.rand(N, W, generator=g) * 4
    check(logits, scores, k)
    fin = (torch.rand(N, W, generator=g) < 0.3).int()
    check(logits, scores, k, fin, eos=V // 2)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [40, 3000, 70000])
def test_ties(V, dtype):
    """Equal values: the lowest beam, then the lowest token. Ties of every size."""
    g = torch.Generator().manual_seed(1)
    for levels in (1, 2, 30):
        say("ties", V, dtype, levels)
        row = torch.randint(0, levels, (1, 1, V), generator=g).to(dtype)
        check(row.expand(2, 4, V).contiguous(), torch.zeros(2, 4), 16)
        check(row.expand(1, 20, V).contiguous(), torch.zeros(1, 20), 64)


@pytest.mark.parametrize("V", [6, 3000, 33000])
def test_slopes(V):
    """Values in order, up and down: all the best ones side by side."""
    up = torch.arange(V, dtype=F)[None, None] * 2.0 ** -7
    check(up.expand(1, 2, V).contiguous(), torch.tensor([[-1.0, -1.5]]), 32)
    check(up.flip(-1).expand(1, 2, V).contiguous(), torch.tensor([[-1.5, -1.0]]), 32)
    block = torch.where(torch.arange(V) % 2048 < 1024, up, up - 1000.0).contiguous()
    check(block, torch.zeros(1, 1), 64)


@pytest.mark.parametrize("V", [50, 5000])
def test_masked_and_other_values(V):
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(2)
    x = normal(g, (1, 8, V), F)
    x[0, 0] = -inf                       # nothing left
    x[0, 1, 3:] = -inf                   # three continuations
    x[0, 2, 5] = nan
    x[0, 3, 6] = inf
    x[0, 4] = torch.finfo(F).min         # the type's lowest value everywhere: V equal ones
    x[0, 5, 1:] = torch.finfo(F).min     # ... but one
    scores = torch.tensor([[0.0, -1.0, 0.0, 0.0, -3.0, -2.0, -inf, -0.5]])
    check(x, scores, 30)
    scores[0, 7] = nan
    check(x, scores, 30)
    scores[0, 4:6] = inf
    check(x, scores, 30)                 # three continuations in all
    check(x[:, :1].contiguous(), torch.zeros(1, 1), 4)
    for t in (BF, H16):
        y = normal(g, (2, 3, V), t)
        y[:, 1] = torch.finfo(t).min
        y[1, 2, ::2] = -inf
        check(y, torch.zeros(2, 3), 20)
    fin = torch.ones(1, 8, dtype=torch.int32)
    check(x, scores, 10, fin, eos=V - 1)  # all have ended (their logits are not read)


def test_scores_in_place_and_first_step():
    """Beams that start alike: only the first counts, with -infinity for the others."""
    g = torch.Generator().manual_seed(3)
    x = normal(g, (4, 1, 3000), F).expand(4, 5, 3000).contiguous()
    scores = torch.full((4, 5), float("-inf"))
    scores[:, 0] = 0
    check(x, scores, 5)
    want = pl.beam(x, scores, 5)
    s, t, p = gpu(scores), ints([[0] * 5] * 4), ints([[0] * 5] * 4)
    kda.beam_select(gpu(x), s, t, p, s)
    assert t.tolist() == want[0] and bool(torch.isfinite(s).all())


def test_workspace_streams_and_graphs():
    g = torch.Generator().manual_seed(4)
    x, scores = gpu(normal(g, (6, 8, 30000), BF, 3.0)), gpu(-torch.rand(6, 8, generator=g))
    want = select(x, scores, 8)
    ws = torch.full((kda.beam_workspace_size(6, 8, 30000, 8),), 255, dtype=torch.uint8, device=dev())
    got = select(x, scores, 8, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = select(x, scores, 8)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    t, p, s = got
    pool = gpu(normal(g, (2, 60, 100), F))
    slots, new = ints(torch.randperm(60, generator=g)[:48].reshape(6, 8).tolist()), ints([[0] * 8] * 6)

    def step():
        kda.beam_select(x, scores, t, p, s, workspace=ws)
        kda.cache_reorder(pool, slots, p, new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(x.roll(17, -1).roll(1, 1))
        before = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (t, p, s, new, pool)]
        pool.copy_(before)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (t, p, s, new, pool))), k
        n, after = pl.reorder(before.cpu(), slots.tolist(), p.tolist())
        assert new.tolist() == n and torch.equal(pool.cpu(), after)


@pytest.mark.parametrize("slot,dtype", [((4,), F), ((7,), BF), ((3,), torch.int8), ((129, 33), F), ((2, 64, 64), BF), ((1001,), torch.uint8)],
                         ids=str)
@pytest.mark.parametrize("L,N,W", [(1, 1, 1), (2, 3, 4), (1, 5, 7), (3, 2, 64)])
def test_reorder(slot, dtype, L, N, W):
    say("reorder", slot, dtype, L, N, W)
    g = torch.Generator().manual_seed(W)
    S = N * W + 5
    pool = torch.randint(-100, 100, (L, S, *slot), generator=g).to(dtype)
    slots = torch.randperm(S, generator=g)[:N * W].reshape(N, W).tolist()
    for kind in range(4):
        if kind == 0:
            parents = torch.randint(0, W, (N, W), generator=g).tolist()
        elif kind == 1:
            parents = [[W - 1 - j for j in range(W)] for _ in range(N)]
        elif kind == 2:
            parents = [[W // 2] * W for _ in range(N)]
        else:
            parents = torch.randint(-2, W + 2, (N, W), generator=g).tolist()
            slots[0][0] = -5
            slots[-1][-1] = S + 3
        n, after = pl.reorder(pool, slots, parents)
        p, new = gpu(pool), torch.full((N, W), -99, dtype=torch.int32, device=dev())
        kda.cache_reorder(p, ints(slots), ints(parents), new)
        assert new.tolist() == n, kind
        assert torch.equal(p.cpu(), after), kind


def test_refusals():
    x, s = torch.zeros(2, 3, 50, device=dev()), torch.zeros(2, 3, device=dev())
    i = ints([[0] * 3] * 2)
    for bad in (dict(scores=s[:1]), dict(tokens=i[0]), dict(parents=i[:, :2]), dict(new_scores=s.to(BF)), dict(finished=s), dict(logits=s)):
        a = dict(logits=x, scores=s, tokens=i, parents=i.clone(), new_scores=s.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            kda.beam_select(**a)
    with pytest.raises(kda.KDAError):
        kda.beam_select(x, s, i, i, s.clone())
    with pytest.raises(kda.KDAError):
        kda.beam_select(x, s, i, i.clone(), s.clone(), finished=i.clone(), eos=50)
    pool = torch.zeros(1, 8, 4, device=dev())
    with pytest.raises(kda.KDAError):
        kda.cache_reorder(pool, i, i.clone(), i)
    with pytest.raises(ValueError):
        kda.cache_reorder(pool, i, i[:1], i.clone())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [50, 9000, 200000])
def test_masked_tokens_add_nothing(V, dtype):
    """A beam that has one token left (a forced one) goes on at its score as it is, as a finished beam
    does: of equal scores the lowest beam comes first, wherever its token is."""
    say("forced", V, dtype)
    for low in (float("-inf"), torch.finfo(dtype).min, -2.0 ** 15):
        x = torch.full((3, 6, V), low)
        for n in range(3):
            for b, v in enumerate((V // 2, V - 1, 0, 7, V // 3, V // 5)):
                x[n, b, v] = (0.0, 5.0, -3.0)[n]
        scores = torch.tensor([-1.5, -0.25, -7.0])[:, None].expand(3, 6).contiguous()
        check(x.to(dtype), scores, 6)
        for fin in ([0, 0, 0, 0, 0, 1], [0, 0, 1, 0, 1, 0], [1, 0, 0, 0, 0, 0]):
            check(x.to(dtype), scores, 6, torch.tensor([fin] * 3, dtype=torch.int32), eos=V // 7)
        # two tokens left, alike: half of the beam's probability each
        for n in range(3):
            for b, v in enumerate((3, 11, V - 2, 21, 20, 30)):
                x[n, b, v] = (0.0, 5.0, -3.0)[n]
        check(x.to(dtype), scores, 12)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [2, 3000, 70000])
def test_zeros_of_both_signs_are_equal(V, dtype):
    """-0.0 and +0.0 are one value: within a piece, across pieces, for either way of cutting a row into
    pieces (few rows and many), and as a finished beam's score."""
    say("zeros", V, dtype)
    g = torch.Generator().manual_seed(V)
    x = torch.zeros(2, 4, V)
    x[..., :5] = -0.0
    check(x.to(dtype), torch.zeros(2, 4), min(4, V))
    x = torch.where(torch.rand(2, 4, V, generator=g) < 0.5, -0.0, 0.0)
    check(x.to(dtype), torch.zeros(2, 4), 16)
    x = torch.where(torch.rand(1, 20, V, generator=g) < 0.01, 0.0, -0.0)   # mostly negative ones
    check(x.to(dtype), torch.zeros(1, 20), 64)
    scores = torch.zeros(2, 4)
    scores[:, 0], scores[1, 2] = -0.0, -0.0
    x = torch.full((2, 4, V), float("-inf"))
    x[..., V // 2] = -0.0                # a sure token: its score is the beam's
    for fin in ([1, 1, 1, 1], [1, 0, 1, 0], [0, 1, 0, 1]):
        check(x.to(dtype), scores, 4, torch.tensor([fin] * 2, dtype=torch.int32), eos=V - 1)
    if V == 3000:
        check(torch.where(torch.rand(72, 8, V, generator=g) < 0.5, -0.0, 0.0).to(dtype), torch.zeros(72, 8), 4)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [60, 3000, 33000])
def test_logits_that_a_score_swallows(V, dtype):
    """Scores beside which logits are lost, as beams that do not count have them at a first step: their
    continuations are equal, so the lowest tokens come first, not those of the largest logits."""
    say("swallowed", V, dtype)
    g = torch.Generator().manual_seed(V + 1)
    x = normal(g, (2, 4, V), dtype, 3.0)
    x[:, 0, 2:] = float("-inf")              # two live continuations, the others are of the beams after it
    x[1, 1, :40] = float("-inf")
    for far in (torch.finfo(F).min, -1e30, -2.0 ** 70):
        scores = torch.full((2, 4), far)
        scores[:, 0] = 0.0
        check(x, scores, 8)
        check(x, scores, 64)
        fin = torch.tensor([[0, 0, 1, 0]] * 2, dtype=torch.int32)
        check(x, scores, 50, fin, eos=V - 1)
    # some of them lost: steps of 2^-12 at a score of 2^40
    scores = torch.full((2, 4), -2.0 ** 40)
    scores[:, 0] = 0.0
    y = (x.float() * 2.0 ** -13).to(dtype)
    y[x == float("-inf")] = float("-inf")
    check(y, scores, 20)
    # logits far below the sum's last bit, and most of them so
    tiny = normal(g, (2, 3, V), F, 2.0 ** -80).to(BF if dtype == H16 else dtype)
    check(tiny, torch.full((2, 3), -1.0), 16)
    tiny[:, :, ::7] = 1.0
    check(tiny, torch.full((2, 3), -1.0), 64)
    # the last piece's and the first token's
    tiny = torch.full((1, 2, V), -5.0, dtype=dtype)
    tiny[0, :, V - 1], tiny[0, 1, V - 9], tiny[0, 0, 0] = 1e-7, 0.0, 1e-7
    check(tiny, torch.tensor([[-2.0 ** 40, -2.0 ** 40]]), 3)
