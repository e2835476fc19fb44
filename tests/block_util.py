"""Shared by the tests of the norm, the gated products and the embedding."""
import numpy as np
import torch

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# A rounding to the type is off by at most half a step: 24, 8 and 11 significand bits.
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 1e-38, BF16: 1e-38, F16: 2.0 ** -25}
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(seed, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen(seed)) * scale).to(dtype)


def whole(seed, *shape, dtype=F32, most=3):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=gen(seed)).to(dtype)


def padded(t, pad):
    """The same values with `pad` values between the rows (NaN) and the base moved by `pad` values."""
    if not pad:
        return t
    flat = torch.full((t[..., 0].numel() * (t.shape[-1] + pad) + pad,), float("nan") if t.is_floating_point() else 77,
                      dtype=t.dtype, device=t.device)
    strides, s = [], t.shape[-1] + pad
    for n in reversed(t.shape[:-1]):
        strides.append(s)
        s *= n
    v = flat.as_strided(t.shape, tuple(reversed(strides)) + (1,), pad)
    v.copy_(t)
    return v


def between(v, pad):
    """What lies between the rows of padded()'s result, which no call may write."""
    base = v.as_strided((v.shape[0], pad), (v.stride(0), 1), v.storage_offset() - pad)
    return base.clone()


def close(got, ref, err, what=""):
    """|got - ref| <= half a step of got's type of |ref| + err, every value; NaN counts as wrong."""
    got64 = got.double()
    tol = ROUND[got.dtype] * ref.abs() + err + TINY[got.dtype]
    bad = ~((got64 - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}: " \
                          f"{got64[bad][0].item()} for {ref[bad][0].item()}, {tol.expand_as(ref)[bad][0].item()} allowed"


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
