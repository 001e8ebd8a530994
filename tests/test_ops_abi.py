"""Refusals of the operators beside kda_fwd, without a GPU: every argument that the header
rules out is reported with its status before anything is launched (fake device pointers are
never dereferenced), sizes are as documented, and the Python wrappers check what they can."""
import ctypes
import os
import re

import pytest
import torch

import gated_delta_rule_87_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ENULL, ESHAPE, EDTYPE, EVALUE, EALIGN, EWS, EHIP, ECAP = range(9)
A = 0x10000000


def fake(i):
    return A + (i << 24)


def call(name, defaults, **kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(kda.lib(), name)(*a.values())


def test_signatures_match_the_header():
    """As many arguments as the header declares, and none declared here that is not there."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kda.h")).read(), flags=re.S)
    L = kda.lib()
    for name in ("kda_cache_workspace_size", "kda_cache_copy", "kda_cache_fork", "kda_cache_free", "kda_cache_compact",
                 "kda_fwd_slots", "kda_glr_carry_rows", "kda_glr_workspace_size", "kda_glr_fwd", "kda_glr_bwd",
                 "kda_glr_step", "kda_layernorm_workspace_size", "kda_layernorm_fwd", "kda_layernorm_bwd"):
        m = re.search(r"\b%s\s*\(([^)]*)\)" % name, src)
        assert m, name
        assert len(m.group(1).split(",")) == len(getattr(L, name).argtypes), name


GLR_F = dict(x=fake(1), g=fake(2), y=fake(3), dtype=1, h0=None, h0d=0, hT=None, hTd=0, carry=None, cu=None, N=0, B=2, T=100,
             D=64, ws=fake(9), wsb=1 << 40, stream=None)
GLR_B = dict(x=fake(1), g=fake(2), dy=fake(3), dtype=1, carry=fake(4), h0=None, h0d=0, df=None, dfd=0, dx=fake(5), dg=fake(6),
             d0=None, d0d=0, cu=None, N=0, B=2, T=100, D=64, ws=fake(9), wsb=1 << 40, stream=None)


@pytest.mark.parametrize("name,d", [("kda_glr_fwd", GLR_F), ("kda_glr_bwd", GLR_B)], ids=["fwd", "bwd"])
def test_glr_refusals(name, d):
    go = lambda **kw: call(name, d, **kw)
    third = "y" if name == "kda_glr_fwd" else "dy"
    for k in ("x", "g", third) + (("carry", "dx", "dg") if third == "dy" else ()):
        assert go(**{k: None}) == ENULL, k
        assert go(**{k: d[k] + 2}) == EALIGN, k
    for bad in (dict(B=0), dict(T=-1), dict(D=0), dict(D=(1 << 22) + 1), dict(cu=fake(7), N=2), dict(cu=fake(7), N=0, B=1),
                dict(B=1 << 20, T=1 << 20), dict(B=1 << 62, T=4), dict(T=1 << 62), dict(B=1 << 24, T=1),
                dict(cu=fake(7), N=1 << 24, B=1), dict(T=1 << 29, D=1 << 20)):
        assert go(**bad) == ESHAPE, bad
    assert go(dtype=0) == EDTYPE and go(dtype=4) == EDTYPE and go(dtype=-1) == EDTYPE
    for p, c in ([("h0", "h0d"), ("hT", "hTd")] if third == "y" else [("h0", "h0d"), ("df", "dfd"), ("d0", "d0d")]):
        assert go(**{p: fake(8), c: 0}) == EDTYPE and go(**{p: fake(8), c: 3}) == EDTYPE
        assert go(**{p: None, c: 2}) == ENULL
        assert go(**{p: fake(8) + 4, c: 2}) == EALIGN
    assert go(cu=fake(7) + 4, N=2, B=1) == EALIGN
    if third == "dy":
        assert go(df=fake(8), dfd=2, d0=fake(8), d0d=2) == EVALUE and go(h0=fake(8), h0d=2, d0=fake(8), d0d=2) == EVALUE
    if third == "y":
        assert go(h0=fake(8), h0d=1, hT=fake(8), hTd=2) == EDTYPE
        assert go(carry=fake(8) + 4) == EALIGN
    need = kda.glr_workspace_size(2, 100, 64)
    assert need > 0 and go(ws=None) == EWS and go(wsb=need - 1) == EWS and go(ws=fake(9) + 16) == EALIGN
    # no tokens: the token tensors may be NULL, the checks after them still hold
    null = {k: None for k in ("x", "g", third) + (("carry", "dx", "dg") if third == "dy" else ())}
    assert go(T=0, D=0, **null) == ESHAPE and go(T=0, dtype=9, **null) == EDTYPE


def test_glr_sizes():
    assert kda.glr_carry_shape(1, 8192, 64) == (64, 64) and kda.glr_carry_shape(3, 43, 5) == (2, 5)
    assert kda.glr_carry_shape(1, 0, 5) == (0, 5)
    assert kda.lib().kda_glr_carry_rows(0, 5) == 0 and kda.lib().kda_glr_carry_rows(1, -5) == 0
    for bad in ((0, 10, 4), (1, -1, 4), (1, 10, 0), (1, 10, (1 << 22) + 1), (1 << 30, 1 << 30, 8), (1, 1 << 29, 1 << 20),
                (1, 10, 64, 1 << 24)):
        assert kda.glr_workspace_size(*bad) == 0


STEP = dict(x=fake(1), g=fake(2), y=fake(3), dtype=2, state=fake(4), sd=2, S=8, src=fake(5), dst=fake(6), N=3, D=64, stream=None)


def test_glr_step_refusals():
    go = lambda **kw: call("kda_glr_step", STEP, **kw)
    for k in ("x", "g", "y", "state", "src", "dst"):
        assert go(**{k: None}) == ENULL, k
        assert go(**{k: STEP[k] + 2}) == EALIGN, k
    for bad in (dict(N=-1), dict(N=1 << 24), dict(N=1 << 40), dict(D=0), dict(S=0), dict(S=(1 << 24) + 1)):
        assert go(**bad) == ESHAPE, bad
    assert go(dtype=5) == EDTYPE and go(sd=0) == EDTYPE and go(sd=3) == EDTYPE


def test_fwd_slots_refusals():
    d = dict(q=fake(1), k=fake(2), v=fake(3), g=fake(4), beta=fake(5), scale=0.1, out=fake(6), A=fake(7), dt=fake(8), lb=-5.0,
             state=fake(9), sd=2, S=8, src=fake(10), dst=fake(11), cu=None, N=0, B=2, T=1, H=2, K=128, V=128, flags=7, stream=None)
    go = lambda **kw: call("kda_fwd_slots", d, **kw)
    for k in ("q", "k", "v", "g", "beta", "out", "A", "dt", "state", "src", "dst"):
        assert go(**{k: None}) == ENULL, k
    for k in ("q", "out", "state", "src", "dst"):
        assert go(**{k: d[k] + 2}) == EALIGN, k
    for bad in (dict(K=64), dict(H=0), dict(S=0), dict(S=(1 << 24) + 1), dict(cu=fake(12), N=2), dict(B=0)):
        assert go(**bad) == ESHAPE, bad
    assert go(sd=0) == EDTYPE and go(sd=3) == EDTYPE
    assert go(lb=-6.0) == EVALUE and go(flags=7 | 16) == EVALUE and go(flags=64) == EVALUE and go(scale=float("nan")) == EVALUE


LN_F = dict(x=fake(1), w=fake(2), b=fake(3), eps=1e-5, y=fake(4), dtype=1, mean=fake(5), rstd=fake(6), M=10, D=64, stream=None)
LN_B = dict(dy=fake(1), x=fake(2), w=fake(3), mean=fake(4), rstd=fake(5), dx=fake(6), dtype=1, dw=fake(7), db=fake(8), M=10,
            D=64, ws=fake(9), wsb=1 << 40, stream=None)


def test_layernorm_refusals():
    for name, d, need in (("kda_layernorm_fwd", LN_F, ("x", "y")), ("kda_layernorm_bwd", LN_B, ("dy", "x", "mean", "rstd"))):
        go = lambda **kw: call(name, d, **kw)
        for k in need:
            assert go(**{k: None}) == ENULL, k
        for k in d:
            if isinstance(d[k], int) and d[k] >= A and k not in ("ws", "wsb"):
                assert go(**{k: d[k] + 4}) == EALIGN, k
        for bad in (dict(M=-1), dict(D=0), dict(D=(1 << 24) + 1), dict(M=1 << 50, D=1 << 20)):
            assert go(**bad) == ESHAPE, bad
        assert go(dtype=0) == EDTYPE and go(dtype=4) == EDTYPE
    for eps in (-1e-5, float("nan"), float("inf")):
        assert call("kda_layernorm_fwd", LN_F, eps=eps) == EVALUE
    need = kda.layernorm_workspace_size(10, 64)
    assert need > 0 and need % 256 == 0
    assert call("kda_layernorm_bwd", LN_B, ws=None) == EWS and call("kda_layernorm_bwd", LN_B, wsb=need - 1) == EWS
    assert call("kda_layernorm_bwd", LN_B, ws=fake(9) + 16) == EALIGN
    # nothing wanted: nothing launched
    assert call("kda_layernorm_bwd", LN_B, dx=None, dw=None, db=None, ws=None, wsb=0) == OK
    # two fp32 rows of D per part, few parts for the widest rows
    assert kda.layernorm_workspace_size(1 << 20, 128) == 2 * 1024 * 128 * 4
    assert kda.layernorm_workspace_size(1 << 20, 8192) == 2 * 256 * 8192 * 4
    assert kda.layernorm_workspace_size(1 << 20, 1 << 24) == 2 * (1 << 24) * 4
    assert kda.layernorm_workspace_size(-1, 5) == 0 and kda.layernorm_workspace_size(5, 0) == 0


def test_cache_refusals():
    pool = dict(pool=fake(1), L=2, S=8, size=64)
    copy = dict(pool, src=fake(2), dst=fake(3), n=4, stream=None)
    fork = dict(pool, used=fake(4), src=fake(2), dst=fake(3), n=4, stream=None)
    comp = dict(pool, used=fake(4), remap=fake(5), table=fake(6), n=4, ws=fake(7), wsb=1 << 20, stream=None)
    for name, d, req in (("kda_cache_copy", copy, ("pool", "src", "dst")),
                         ("kda_cache_fork", fork, ("pool", "used", "src", "dst")),
                         ("kda_cache_compact", comp, ("pool", "used", "remap"))):
        go = lambda **kw: call(name, d, **kw)
        for k in req:
            assert go(**{k: None}) == ENULL, (name, k)
            assert go(**{k: d[k] + 2}) == EALIGN, (name, k)
        for bad in (dict(L=0), dict(S=0), dict(S=(1 << 24) + 1), dict(size=0), dict(n=-1), dict(n=1 << 31),
                    dict(L=1 << 40), dict(L=1 << 20, S=1 << 20, size=1 << 30)):
            assert go(**bad) == ESHAPE, (name, bad)
    assert call("kda_cache_compact", comp, table=fake(6) + 2) == EALIGN
    for bad in (dict(dst=fork["src"]), dict(dst=fork["used"]), dict(src=fork["used"])):
        assert call("kda_cache_fork", fork, **bad) == EVALUE, bad
    for bad in (dict(remap=comp["used"]), dict(table=comp["used"]), dict(table=comp["remap"])):
        assert call("kda_cache_compact", comp, **bad) == EVALUE, bad
    need = kda.lib().kda_cache_workspace_size(8)
    assert call("kda_cache_compact", comp, ws=None) == EWS and call("kda_cache_compact", comp, wsb=need - 1) == EWS
    assert call("kda_cache_compact", comp, ws=fake(7) + 16) == EALIGN
    free = dict(used=fake(4), S=8, slots=fake(2), n=4, stream=None)
    for bad, rc in ((dict(used=None), ENULL), (dict(slots=None), ENULL), (dict(S=0), ESHAPE), (dict(n=-1), ESHAPE),
                    (dict(used=fake(4) + 1), EALIGN), (dict(slots=fake(2) + 1), EALIGN)):
        assert call("kda_cache_free", free, **bad) == rc, bad
    # no requests: nothing is launched
    assert call("kda_cache_copy", copy, n=0, src=None, dst=None) == OK
    assert call("kda_cache_fork", fork, n=0, src=None, dst=None) == OK
    assert call("kda_cache_free", free, n=0, slots=None) == OK
    assert kda.lib().kda_cache_workspace_size(0) == 0 and kda.lib().kda_cache_workspace_size((1 << 24) + 1) == 0


def test_python_wrappers_refuse_cpu_tensors():
    x, i = torch.zeros(2, 3, 8), torch.zeros(3, dtype=torch.int32)
    for f in (lambda: kda.glr_fwd(x, x, x), lambda: kda.glr_bwd(x, x, x, x, x, x), lambda: kda.glr_step(x[0], x[0], x[0], x[0], i, i),
              lambda: kda.layernorm_fwd(x, None, None, 1e-5, x), lambda: kda.layernorm_bwd(x, x, None, x, x, x),
              lambda: kda.cache_copy(x, i, i), lambda: kda.cache_fork(x, i, i, i), lambda: kda.cache_free(i, i),
              lambda: kda.cache_compact(x, i, i)):
        with pytest.raises(ValueError):
            f()


def test_no_operator_kernel_uses_scratch(tmp_path):
    """No spills and no private memory in the operators' kernels."""
    from test_sources import _device_asm
    for src in ("kda_glr.hip", "kda_layernorm.hip", "kda_cache.hip"):
        text = "\n".join(_device_asm(src, tmp_path))
        spills = [int(v) for v in re.findall(r"\.vgpr_spill_count:\s+(\d+)", text)]
        priv = [int(v) for v in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)]
        assert spills and not any(spills) and not any(priv), (src, spills, priv)


def test_states_of_a_cache_layer_are_accepted():
    """A state begins where a layer of a cache [L, S, D] can: at any element where rows are no
    whole vectors, at a vector's elements (8 bytes of bf16 beside fp32 tokens) where they are."""
    for dtype, sd, D, unit in ((2, 2, 129, 4), (1, 1, 129, 2), (1, 2, 12, 4), (3, 1, 100, 2), (2, 1, 7, 2), (2, 1, 12, 8),
                               (2, 2, 12, 16), (1, 1, 64, 16), (1, 2, 64, 16)):
        go = lambda off: call("kda_glr_step", STEP, dtype=dtype, sd=sd, D=D, N=0, state=fake(4) + off)   # N = 0: no launch
        assert go(unit) == OK and go(unit // 2) == EALIGN, (dtype, sd, D)
        for name, d, states in (("kda_glr_fwd", GLR_F, (("h0", "h0d"), ("hT", "hTd"))),
                                ("kda_glr_bwd", GLR_B, (("h0", "h0d"), ("df", "dfd"), ("d0", "d0d")))):
            for p, c in states:
                go = lambda off: call(name, d, dtype=dtype, D=D, ws=None, **{p: fake(8) + off, c: sd})   # refused after it
                assert go(unit) == EWS and go(unit // 2) == EALIGN, (name, p, dtype, sd, D)


def test_flags_given_as_the_slots_to_free_are_refused():
    """kda_cache_free writes used while it reads slots: one array for both would be a race."""
    free = dict(used=fake(4), S=8, slots=fake(4), n=4, stream=None)
    assert call("kda_cache_free", free) == EVALUE
    assert call("kda_cache_free", free, n=0) == OK   # nothing is done
