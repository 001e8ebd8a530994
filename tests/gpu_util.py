"""What the GPU tests of a state space layer's operators share."""
import torch

BF, H16, F = torch.bfloat16, torch.float16, torch.float32
DTYPES = [BF, H16, F]


def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def say(*a):
    print("[gpu-test]", *a, flush=True)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def gpu(t):
    return None if t is None else t.to(dev())


def normal(g, shape, dtype=F, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def blank(shape, dtype=F):
    """An output that holds NaN until it is written."""
    return torch.full(shape, float("nan"), dtype=dtype, device=dev())


def cu_of(bounds):
    return None if bounds is None else torch.tensor(bounds, dtype=torch.int64, device=dev())


def spans_of(bounds, B, T):
    if bounds is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return list(zip(bounds[:-1], bounds[1:]))


def covered(sp, tokens):
    m = torch.zeros(tokens, dtype=torch.bool)
    for lo, hi in sp:
        m[lo:hi] = True
    return m


def untouched(name, got, rows):
    """Tokens that no sequence covers are as they were: NaN."""
    assert bool(torch.isnan(got[~rows].float()).all()), name


def same(a, b):
    """The same bits, NaN included."""
    return torch.equal(torch.nan_to_num(a.float(), nan=-7.75e30), torch.nan_to_num(b.float(), nan=-7.75e30))
