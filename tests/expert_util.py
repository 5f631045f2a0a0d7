"""Inputs, 64-bit definitions and error bounds for the tests of the 8-bit
linear layers and the experts' operators.

Bounds count roundings.  A rounding to a type t is off by at most
finfo(t).eps / 2 of the value (H below), or by half the smallest subnormal
(TINY) where that is larger.  A sum of n fp32 terms in any order is off by at
most n * 2^-23 of the sum of their magnitudes (2^-23 and not 2^-24 per
addition: the tensor cores' adders may truncate).
"""
import torch

H = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def pitched(shape, dtype, device="cuda", extra=0):
    """Zeros of `shape` whose row pitch is a multiple of 16 bytes (plus
    `extra` such units): a strided view for odd widths."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = max(1, -(-shape[-1] // per) + extra) * per
    return torch.zeros(*shape[:-1], ld, dtype=dtype, device=device)[..., :shape[-1]]


def normal(shape, dtype, seed, scale=1.0, device="cuda", extra=0):
    g = torch.Generator().manual_seed(seed)
    out = pitched(shape, dtype, device, extra)
    out.copy_((torch.randn(shape, generator=g) * scale).to(dtype))
    return out


def ints8(shape, seed, lo=-128, hi=128, device="cuda", extra=0):
    g = torch.Generator().manual_seed(seed)
    out = pitched(shape, torch.int8, device, extra)
    out.copy_(torch.randint(lo, hi, shape, generator=g, dtype=torch.int8))
    return out


def positive(shape, seed, lo=0.5, hi=1.5, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(shape, generator=g) * (hi - lo) + lo).to(device)


def offsets_of(counts, device="cuda"):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return o.to(device)


def close(got, ref, bound, what=""):
    """|got - ref| <= bound elementwise; ref and bound in float64."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
                             f"got {got[i].item()}, want {ref[i].item()}, bound {bound[i].item()}")


def product16(A, W, dtype):
    """A @ W in 64 bits, and the bound of an fp32 sum rounded once to dtype."""
    a, w = A.double(), W.double()
    ref = a @ w
    return ref, H[dtype] * ref.abs() * 1.01 + TINY[dtype] + a.shape[1] * 2.0 ** -23 * (a.abs() @ w.abs())


def product8(A, rs, W, cs, dtype):
    """The exact integer sum times both scales, and the bound: the sum to
    fp32, two products in fp32, one rounding to dtype."""
    ref = (A.double() @ W.double()) * rs.double()[:, None] * cs.double()
    return ref, ref.abs() * (H[dtype] * 1.01 + 4 * 2.0 ** -24) + TINY[dtype]
