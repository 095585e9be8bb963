"""What the tests of the operators around the half layer share: inputs, and bounds
in half steps of the types."""
import math

import torch

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24                                             # half a step of fp32
# smallest step of a result, for values below the normal range
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -133, F32: 2.0 ** -149}
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


def half_step(t):
    return torch.finfo(t).eps / 2


def rnd(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda")


def ints(seed, lo, hi, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda")


def close(got, ref, slack):
    """|got - ref| <= one rounding of ref to got's type + slack, everywhere."""
    assert got.shape == ref.shape
    err = (got.to(F64) - ref).abs()
    bound = half_step(got.dtype) * (ref.abs() + slack) + slack + TINY[got.dtype]
    over = ref.to(got.dtype)                    # a value past the type's range rounds to an infinity
    bad = ~((err <= bound) | (over.isinf() & (got == over)))
    if bad.any():
        at = bad.nonzero()[:4]
        raise AssertionError("%d of %d off, first at %s: %s, not %s (bound %s)" % (
            int(bad.sum()), bad.numel(), at.tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist(),
            (bound + torch.zeros_like(ref))[bad][:4].tolist()))


def strided(t, pad):
    """t with rows `pad` elements further apart than they are long, NaN between them."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def shifted(t):
    """t one element past an aligned address."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


def act_ref(z, act):
    """Value and slope of an activation."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).to(F64)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * torch.sigmoid(-c * (z + 0.044715 * z ** 3)) * c * (1 + 0.134145 * z * z)
