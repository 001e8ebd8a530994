"""Caches of states on the GPU: slots copied, forked, freed and compacted against plain lists,
KDA steps on a cache's slots against kda_fwd_recurrent, and a run of the operators together."""
import pytest
import torch

import kda_inputs
import gated_delta_rule_87_amd as kda
import plain_ops as po

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def say(*a):
    print("[gpu-test]", *a, flush=True)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def make_pool(L, S, slot, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-100, 100, (L, S, *slot), generator=gen).to(dtype)


def flags(S, share, seed):
    return (torch.rand(S, generator=torch.Generator().manual_seed(seed)) < share).int().tolist()


SLOTS = [((4,), F), ((7,), BF), ((3,), torch.int8), ((128, 33), F), ((2, 128, 128), BF), ((1001,), torch.uint8)]


@pytest.mark.parametrize("slot,dtype", SLOTS, ids=[f"{s}-{str(d)[6:]}" for s, d in SLOTS])
@pytest.mark.parametrize("L,S", [(1, 1), (2, 9), (3, 50)])
def test_copy(slot, dtype, L, S):
    say("copy", slot, dtype, L, S)
    pool = make_pool(L, S, slot, dtype)
    perm = torch.randperm(S, generator=torch.Generator().manual_seed(S)).tolist()
    half = S // 2
    src, dst = [perm[i % max(1, half)] for i in range(S - half)], perm[half:]   # a source may be named twice
    if S == 1:
        src, dst = [0], [0]
    src, dst = src + [-1, 0, S, 2 ** 31 - 1], dst + [0, -1, 0, 0]   # pairs that do nothing
    want = pool.clone()
    for a, b in zip(src[:-4], dst[:-4]):
        want[:, b] = pool[:, a]
    p = pool.to(dev())
    kda.cache_copy(p, ints(src), ints(dst))
    assert torch.equal(p.cpu(), want)


@pytest.mark.parametrize("slot,dtype", SLOTS[:5:2], ids=[f"{s}" for s, d in SLOTS[:5:2]])
@pytest.mark.parametrize("S,n,share", [(1, 1, 0.0), (1, 3, 1.0), (10, 4, 0.5), (40, 40, 0.3), (1500, 300, 0.7), (3000, 2500, 0.5), (64, 1, 1.0)])
def test_fork_and_free(slot, dtype, S, n, share):
    if S > 100 and len(slot) > 1:
        slot = (16,)
    say("fork", slot, dtype, S, n, share)
    L = 2
    pool, used = make_pool(L, S, slot, dtype, seed=1), flags(S, share, S)
    gen = torch.Generator().manual_seed(n)
    live = [i for i in range(S) if used[i]]
    src = [live[int(i)] if live else -1 for i in torch.randint(0, max(1, len(live)), (n,), generator=gen)]
    if n > 3:
        src[1], src[2], src[3] = -1, -7, S
        free = [i for i in range(S) if not used[i]]
        if free:
            src[0] = free[-1]   # not a used slot before the call
    dst, after = po.fork(used, src)
    want = pool.clone()
    for a, b in zip(src, dst):
        if b >= 0:
            want[:, b] = pool[:, a] if a >= 0 else 0
    p, u, d = pool.to(dev()), ints(used), torch.full((n,), -99, dtype=torch.int32, device=dev())
    kda.cache_fork(p, u, ints(src), d)
    assert d.tolist() == dst and u.tolist() == after
    assert torch.equal(p.cpu(), want)
    gone = [s for s in dst if s >= 0][::2]
    kda.cache_free(u, ints(gone + gone + [-1, S, S + 100]))
    for s in gone:
        after[s] = 0
    assert u.tolist() == after


@pytest.mark.parametrize("slot,dtype", SLOTS, ids=[f"{s}-{str(d)[6:]}" for s, d in SLOTS])
@pytest.mark.parametrize("S,share", [(1, 0.0), (1, 1.0), (2, 0.5), (33, 0.5), (200, 0.1), (200, 0.95)])
def test_compact(slot, dtype, S, share):
    say("compact", slot, dtype, S, share)
    check_compact(slot, dtype, S, flags(S, share, S + 3), 2)


@pytest.mark.parametrize("S", [1023, 1024, 1025, 5000, 70000])
def test_compact_many_slots(S):
    say("compact", S, "slots")
    check_compact((4,), BF, S, flags(S, 0.6, S), 1)


@pytest.mark.parametrize("used", [[0, 0, 0, 1, 1], [1, 1, 0, 0, 0], [0, 1, 0, 1, 0], [0] * 6, [1] * 6, [0, 0, 0, 0, 1], [0, 5, -1, 0]])
def test_compact_patterns(used):
    check_compact((5,), F, len(used), used, 1)


def check_compact(slot, dtype, S, used, L):
    pool = make_pool(L, S, slot, dtype, seed=2)
    moves, remap = po.compact([int(u != 0) for u in used])
    want = pool.clone()
    for a, b in moves:
        want[:, b] = pool[:, a]
    table = [S - 1 - i for i in range(S)] + [-1, S, -5, 2 ** 31 - 1]
    p, u, r, t = pool.to(dev()), ints(used), torch.full((S,), -99, dtype=torch.int32, device=dev()), ints(table)
    kda.cache_compact(p, u, r, table=t)
    n = sum(1 for x in used if x)
    assert r.tolist() == remap
    assert u.tolist() == [1] * n + [0] * (S - n)
    assert t.tolist() == [remap[s] if 0 <= s < S else -1 for s in table]
    assert torch.equal(p.cpu(), want)


def test_nothing_to_do():
    say("n = 0")
    e = torch.empty(0, dtype=torch.int32, device=dev())
    p, u = torch.ones(1, 3, 8, device=dev()), ints([1, 0, 1])
    kda.cache_copy(p, e, e)
    kda.cache_fork(p, u, e, e)
    kda.cache_free(u, e)
    assert (p == 1).all() and u.tolist() == [1, 0, 1]


def test_slots_past_32_bits():
    """A cache of more than 2^32 bytes whose last slots are forked and moved."""
    say("a cache of 6 GiB")
    S = 3 * 512
    p = torch.zeros(1, S, 1 << 20, dtype=F, device=dev())
    p[0, S - 1] = 5
    p[0, S - 2, -1] = 3
    used = ints([0] * (S - 2) + [1, 1])
    dst = torch.empty(1, dtype=torch.int32, device=dev())
    kda.cache_fork(p, used, ints([S - 1]), dst)
    assert dst.tolist() == [0] and bool((p[0, 0] == 5).all())
    remap = torch.empty(S, dtype=torch.int32, device=dev())
    kda.cache_compact(p, used, remap)
    assert remap[S - 2:].tolist() == [1, 2] and float(p[0, 1, -1]) == 3 and bool((p[0, 2] == 5).all())


def test_graph_of_a_turn():
    """Fork, step and free captured into a graph and replayed, against eager calls."""
    say("graph of fork and free")
    S, n = 40, 6
    used0 = flags(S, 0.4, 9)
    live = [i for i in range(S) if used0[i]]
    p, u = make_pool(2, S, (300,), F, seed=3).to(dev()), ints(used0)
    src, dst = ints([live[i % len(live)] for i in range(n)]), torch.empty(n, dtype=torch.int32, device=dev())
    x, g, y = torch.randn(n, 300, device=dev()), -torch.rand(n, 300, device=dev()), torch.empty(n, 300, device=dev())

    def turn(p, u, dst, y):
        kda.cache_fork(p, u, src, dst)
        kda.glr_step(x, g, y, p[1], dst, dst)
        kda.cache_free(u, dst[:3])

    turn(p.clone(), u.clone(), dst, y)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        turn(p, u, dst, y)
    pe, ue, de, ye = p.clone(), u.clone(), dst.clone(), y.clone()
    for rep in range(4):
        src.copy_(ints([live[(i + rep) % len(live)] for i in range(n)]))
        x.normal_()
        gr.replay()
        turn(pe, ue, de, ye)
        torch.cuda.synchronize()
        assert torch.equal(p, pe) and torch.equal(u, ue) and torch.equal(dst, de) and torch.equal(y, ye), rep


# ---- KDA on slots -----------------------------------------------------------------


def kda_args(lengths, H, seed, device):
    w = kda_inputs.custom(lengths=lengths, H=H, state='fp32')
    w.seed = seed
    d = kda_inputs.make_inputs(w)
    return {k: (v.to(device) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


@pytest.mark.parametrize("state", [F, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("lengths,H", [([1], 1), ([1, 1, 1, 1, 1], 8), ([3, 0, 1, 20], 2), ([1] * 40, 4)])
def test_kda_on_slots(state, lengths, H):
    """The same bits as kda_fwd_recurrent on the states gathered from the slots."""
    say("kda on slots", state, len(lengths), H)
    d = dev()
    x = kda_args(lengths, H, 5, d)
    n = len(lengths)
    S = 2 * n + 2
    pool = (torch.randn(S, H, 128, 128, generator=torch.Generator().manual_seed(1)) * 0.02).to(state).to(d)
    perm = torch.randperm(S, generator=torch.Generator().manual_seed(2)).tolist()
    src, dst = perm[:n], perm[n:2 * n]
    if n > 3:
        src[1], src[2], dst[3] = -1, src[0], S
    dst[0] = src[0] if n == 1 else dst[0]
    h0 = torch.stack([pool[s] if 0 <= s < S else torch.zeros_like(pool[0]) for s in src])
    T = sum(lengths)
    o_ref, f_ref = torch.empty(1, T, H, 128, dtype=BF, device=d), torch.empty_like(h0)
    args = [x[k] for k in ("q", "k", "v", "g", "beta", "scale")]
    rest = [x["A_log"], x["dt_bias"], x["lower_bound"]]
    kda.fwd_recurrent(*args, o_ref, *rest, initial_state=h0, final_state=f_ref, cu_seqlens=x["cu_seqlens"])
    want = pool.clone()
    for i, s in enumerate(dst):
        if 0 <= s < S:
            want[s] = f_ref[i]
    out = torch.empty_like(o_ref)
    kda.fwd_slots(*args, out, *rest, pool, ints(src), ints(dst), cu_seqlens=x["cu_seqlens"])
    torch.cuda.synchronize()
    assert torch.equal(out, o_ref) and torch.equal(pool, want)


def test_kda_on_slots_rows_and_switches():
    """Rows without cu_seqlens, and the unbounded gate: the flags reach the kernel."""
    d = dev()
    w = kda_inputs.custom(B=3, T=4, H=2, state='fp32')
    x = {k: (v.to(d) if isinstance(v, torch.Tensor) else v) for k, v in kda_inputs.make_inputs(w).items()}
    pool = torch.cat([x["initial_state"], torch.zeros_like(x["initial_state"])])
    args = [x[k] for k in ("q", "k", "v", "g", "beta", "scale")]
    rest = [x["A_log"], x["dt_bias"], x["lower_bound"]]
    o, f = torch.empty_like(x["v"]), torch.empty_like(x["initial_state"])
    kda.fwd_recurrent(*args, o, *rest, initial_state=x["initial_state"], final_state=f, safe_gate=False)
    o2 = torch.empty_like(o)
    kda.fwd_slots(*args, o2, *rest, pool, ints([0, 1, 2]), ints([3, 4, 5]), safe_gate=False)
    assert torch.equal(o, o2) and torch.equal(pool[3:], f) and torch.equal(pool[:3], x["initial_state"])


def test_operators_together():
    """Prefill of two layers' states (KDA and the gated recurrence, its input normed), the states
    in a cache each, prompts forked for samples, some dropped, the cache compacted, and a token
    for each that is left: the same as calls on states that were never moved."""
    say("prefill, norm, fork, free, compact, step")
    d = dev()
    H, lengths = 2, [70, 5, 33]
    D, n = H * 128, 3
    x = kda_args(lengths, H, 6, d)
    T = sum(lengths)
    args = [x[k] for k in ("q", "k", "v", "g", "beta", "scale")]
    rest = [x["A_log"], x["dt_bias"], x["lower_bound"]]
    S = 16
    k_pool, g_pool = torch.zeros(1, S, H, 128, 128, device=d), torch.zeros(1, S, D, device=d)
    used = ints([0] * S)
    first = torch.empty(n, dtype=torch.int32, device=d)
    kda.cache_fork(k_pool, used, ints([-1] * n), first)   # three new sequences
    assert first.tolist() == [0, 1, 2]
    o = torch.empty(1, T, H, 128, dtype=BF, device=d)
    kda.fwd(*args, o, *rest, final_state=k_pool[0, :n], cu_seqlens=x["cu_seqlens"])
    w, b = torch.rand(128, device=d) + 0.5, torch.randn(128, device=d)
    normed = torch.empty_like(o)
    kda.layernorm_fwd(o, w, b, 1e-5, normed)
    gate = -torch.rand(1, T, D, device=d).to(BF)
    y = torch.empty(1, T, D, dtype=BF, device=d)
    kda.glr_fwd(normed.view(1, T, D), gate, y, final_state=g_pool[0, :n], cu_seqlens=x["cu_seqlens"])
    v, _ = po.layernorm(o.cpu().reshape(-1, 128), w.cpu(), b.cpu(), 1e-5)
    v2, e2 = po.glr(normed.cpu().view(T, D), gate.cpu()[0], po.spans(x["cu_seqlens"].cpu(), 1, T))
    po.assert_near("y", y[0], v2["y"], e2["y"])
    # five samples: the slots' numbers are the same in both caches
    picks = [0, 2, 2, 1, 0]
    samples = torch.empty(5, dtype=torch.int32, device=d)
    kda.cache_fork(k_pool, used, ints(picks), samples)
    kda.cache_copy(g_pool, ints(picks), samples)
    assert samples.tolist() == [3, 4, 5, 6, 7]
    kda.cache_free(used, ints([0, 1, 2, 4]))   # the prompts and a sample end
    left = ints([3, 5, 6, 7])
    remap = torch.empty(S, dtype=torch.int32, device=d)
    used2 = used.clone()
    kda.cache_compact(k_pool, used, remap)
    slots = left.clone()
    kda.cache_compact(g_pool, used2, remap, table=slots)
    assert sorted(slots.tolist()) == [0, 1, 2, 3] and used.tolist() == used2.tolist() == [1] * 4 + [0] * 12
    # a token for each, on the slots and on the states kept aside
    t = kda_args([1] * 4, H, 7, d)
    targs = [t[k] for k in ("q", "k", "v", "g", "beta", "scale")]
    trest = [t["A_log"], t["dt_bias"], t["lower_bound"]]
    order = [picks[0], picks[2], picks[3], picks[4]]
    h0, o1 = torch.empty(n, H, 128, 128, device=d), torch.empty_like(o)
    kda.fwd(*args, o1, *rest, final_state=h0, cu_seqlens=x["cu_seqlens"])
    h0 = h0[order].contiguous()
    oa, ob, f = torch.empty_like(t["v"]), torch.empty_like(t["v"]), torch.empty_like(h0)
    kda.fwd_recurrent(*targs, oa, *trest, initial_state=h0, final_state=f, cu_seqlens=t["cu_seqlens"])
    kda.fwd_slots(*targs, ob, *trest, k_pool[0], slots, slots, cu_seqlens=t["cu_seqlens"])
    assert torch.equal(oa, ob)
    assert torch.equal(k_pool[0][slots.long()], f)
    gx, gg = torch.randn(4, D, device=d), -torch.rand(4, D, device=d)
    gy = torch.empty(4, D, device=d)
    kda.glr_step(gx, gg, gy, g_pool[0], slots, slots)
    v3, e3 = po.glr(gx.cpu(), gg.cpu(), [(i, i + 1) for i in range(4)], v2["final"][order])
    po.assert_near("step", gy, v3["y"], e3["y"] + e2["final"][order])


def guarded(need):
    """A workspace of exactly `need` bytes with a guard behind it."""
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=dev())
    return room[:need], room[need:]


@pytest.mark.parametrize("T,D", [(40, 8), (300, 129), (1000, 64), (1025, 7), (5000, 264)])
def test_workspaces_are_not_overrun(T, D):
    """Every operator inside a workspace of the size that it asks for, whatever was in it."""
    say("workspaces of the exact size", T, D)
    d = dev()
    cu = torch.tensor([0, T // 3, T // 3, T], device=d)
    x, g = torch.randn(1, T, D, device=d), -torch.rand(1, T, D, device=d)
    y, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    st, d0, carry = torch.randn(3, D, device=d), torch.empty(3, D, device=d), torch.empty(kda.glr_carry_shape(1, T, D), device=d)
    ws, guard = guarded(kda.glr_workspace_size(1, T, D, 3))
    kda.glr_fwd(x, g, y, initial_state=st, final_state=st, cu_seqlens=cu, carry=carry, workspace=ws)   # states staged there
    assert (guard == 0x5A).all()
    kda.glr_bwd(x, g, y, carry, dx, dg, d_initial=d0, cu_seqlens=cu, workspace=ws)
    assert (guard == 0x5A).all()
    mean, rstd, dw, db = (torch.ones(n, device=d) for n in (T, T, D, D))
    ws, guard = guarded(kda.layernorm_workspace_size(T, D))
    kda.layernorm_bwd(y[0], x[0], None, mean, rstd, dx[0], d_weight=dw, d_bias=db, workspace=ws)
    assert (guard == 0x5A).all()
    ws, guard = guarded(kda.lib().kda_cache_workspace_size(T))
    pool, used, remap = torch.zeros(1, T, 4, device=d), ints([i % 2 for i in range(T)]), ints([0] * T)
    kda.cache_compact(pool, used, remap, workspace=ws)
    assert (guard == 0x5A).all()


@pytest.mark.parametrize("state", [F, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("dtype", [F, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("L,S,D", [(2, 3, 129), (3, 5, 7), (3, 3, 4), (2, 1, 1), (2, 7, 12)])
def test_every_layer_of_a_cache(dtype, state, L, S, D):
    """Layers of a pool [L, S, D] begin at any multiple of their element: steps, and states
    passed to and from the recurrence, on each of them as on a copy."""
    say("layers of odd widths", dtype, state, L, S, D)
    gen = torch.Generator().manual_seed(D)
    d = dev()
    pool = torch.randn(L, S, D, generator=gen).to(state).to(d)
    n = max(1, S // 2)
    src, dst = (torch.arange(k, k + n, dtype=torch.int32, device=d) for k in (0, S - n))
    for layer in range(L):
        x, g = torch.randn(n, D, generator=gen).to(dtype).to(d), -torch.rand(n, D, generator=gen).to(dtype).to(d)
        y, y2 = torch.empty_like(x), torch.empty_like(x)
        want = pool.clone()
        copy = pool[layer].clone()
        kda.glr_step(x, g, y2, copy, src, dst)
        want[layer] = copy
        kda.glr_step(x, g, y, pool[layer], src, dst)
        assert torch.equal(y, y2) and torch.equal(pool, want), layer
    for T in (20, 300):
        x, g = torch.randn(S, T, D, generator=gen).to(dtype).to(d), -torch.rand(S, T, D, generator=gen).to(dtype).to(d)
        for layer in range(1, L):
            fin, other = torch.zeros_like(pool), torch.zeros_like(pool)
            grad, g0 = torch.zeros_like(pool), [torch.empty(S, D, dtype=state, device=d) for _ in range(2)]
            outs = []
            for h0, f, dh, d0 in ((pool[layer], fin[layer], pool[layer - 1], grad[layer]),
                                  (pool[layer].clone(), g0[0], pool[layer - 1].clone(), g0[1])):
                y, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
                carry = torch.empty(kda.glr_carry_shape(S, T, D), device=d)
                kda.glr_fwd(x, g, y, initial_state=h0, final_state=f, carry=carry)
                kda.glr_bwd(x, g, x, carry, dx, dg, initial_state=h0, d_final=dh, d_initial=d0)
                outs.append((y, dx, dg, f, d0))
            assert all(torch.equal(a, b) for a, b in zip(*outs)), (T, layer)
            assert not fin[layer - 1].any() and not grad[layer - 1].any()


def test_outputs_count_their_versions():
    """A tensor that an operator has written counts as changed: autograd refuses to use what it
    had saved of it, instead of taking the new values for the old."""
    say("versions")
    d = dev()
    x, g = torch.randn(1, 40, 16, device=d), -torch.rand(1, 40, 16, device=d)
    new = lambda: torch.zeros_like(x)
    i, st = torch.zeros(1, dtype=torch.int32, device=d), torch.zeros(1, 16, device=d)
    carry = torch.zeros(kda.glr_carry_shape(1, 40, 16), device=d)
    o = {k: new() for k in ("y", "dx", "dg", "n", "dn")}
    v = {k: torch.zeros(40, device=d) for k in ("mean", "rstd")}
    w = {k: torch.zeros(16, device=d) for k in ("dw", "db")}
    pool, used, dst, remap, table = torch.zeros(1, 4, 16, device=d), i.new_zeros(4), i.clone(), i.new_zeros(4), i.clone()
    fin, d0, step = st.clone(), st.clone(), torch.zeros(1, 16, device=d)
    calls = [
        (lambda: kda.glr_fwd(x, g, o["y"], final_state=fin, carry=carry), (o["y"], fin, carry)),
        (lambda: kda.glr_bwd(x, g, x, carry, o["dx"], o["dg"], d_initial=d0), (o["dx"], o["dg"], d0)),
        (lambda: kda.glr_step(x[0, :1], g[0, :1], step, pool[0], i, i), (step, pool)),
        (lambda: kda.layernorm_fwd(x, None, None, 1e-5, o["n"], mean=v["mean"], rstd=v["rstd"]), (o["n"], v["mean"], v["rstd"])),
        (lambda: kda.layernorm_bwd(x, x, None, v["mean"], v["rstd"], o["dn"], d_weight=w["dw"], d_bias=w["db"]), (o["dn"], w["dw"], w["db"])),
        (lambda: kda.cache_fork(pool, used, i - 1, dst), (pool, used, dst)),
        (lambda: kda.cache_copy(pool, i, i + 1), (pool,)),
        (lambda: kda.cache_compact(pool, used, remap, table=table), (pool, used, remap, table)),
        (lambda: kda.cache_free(used, i), (used,))]
    inputs = (x, g, i)
    before = [t._version for t in inputs]
    for n, (call, outs) in enumerate(calls):
        old = [t._version for t in outs]
        call()
        assert all(t._version > k for t, k in zip(outs, old)), n
    assert [t._version for t in inputs] == before
    p = torch.ones(16, device=d, requires_grad=True)
    loss = (o["n"] * p).sum()
    kda.layernorm_fwd(x * 2, None, None, 1e-5, o["n"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        kda.layernorm_fwd(x * 2, None, None, 1e-5, torch.empty_like(x))


def test_two_caches_of_one_numbering():
    """KDA's states and those of a recurrence under the same slot numbers, as the header describes
    it: forked in one cache and copied in the other, where a new sequence begins from slot -1;
    the second cache compacted by the flags from before the first was."""
    say("two caches of one numbering")
    d = dev()
    S, D = 6, 40
    k_pool, g_pool = make_pool(1, S, (3,), F, seed=4).to(d), make_pool(1, S, (D,), F, seed=5).to(d)
    used = ints([0, 1, 0, 1, 0, 1])
    src, dst = ints([3, -1, 5]), ints([0] * 3)
    old = g_pool.clone()
    kda.cache_fork(k_pool, used, src, dst)
    kda.cache_copy(g_pool, src, dst)
    assert dst.tolist() == [0, 2, 4]
    x, g, y = torch.randn(3, D, device=d), -torch.rand(3, D, device=d), torch.empty(3, D, device=d)
    begin = torch.where(src < 0, src, dst)
    kda.glr_step(x, g, y, g_pool[0], begin, dst)
    v, e = po.glr(x.cpu(), g.cpu(), [(i, i + 1) for i in range(3)], torch.stack([old[0, 3], torch.zeros(D, device=d), old[0, 5]]).cpu())
    po.assert_near("y", y, v["y"], e["y"])
    kda.cache_free(used, ints([1, 2]))   # 0, 3, 4 and 5 are left
    flags_before, remap = used.clone(), ints([0] * S)
    before = g_pool.clone()
    kda.cache_compact(k_pool, used, remap)
    kda.cache_compact(g_pool, flags_before, remap)
    assert used.tolist() == flags_before.tolist() == [1, 1, 1, 1, 0, 0] and remap.tolist() == [0, -1, -1, 3, 1, 2]
    assert torch.equal(g_pool[0, :4], before[0, [0, 4, 5, 3]])
